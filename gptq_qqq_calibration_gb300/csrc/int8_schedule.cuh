// Who computes what in the 8-bit integer product on SM pairs: the tiles of
// Y^T = Wq Xq^T, the units a tile's sum is split in, and the pair that takes each.
// Host and device functions, so that the kernel, the host library and a CPU test of
// the schedule (tests/int8_schedule_check.cu) run the same code.
//
// Two ways.  Whole tiles in turn, where there are many; the tiles of the last turn may be
// split along their sums.  Or an even share of all tiles' stages for every pair, where
// there are few tiles: a pair then has a part of a tile at either end of its share, at
// most.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace hk {
namespace i8 {

constexpr int kKB = 128;        // contraction steps of one stage
constexpr int kMaxTok = 192;    // tokens of a tile: the MMA's columns
constexpr int kMaxRows = 128;   // weight rows of a tile per CTA: the MMA's rows
constexpr int kChunk = 8;       // stages whose sums stay below 2^24: 1,024 products of at most 2^14
constexpr int kGroupF = 8;      // row tiles that run side by side (their token boxes meet in L2)
constexpr int kMaxParts = 8;

struct Schedule {
    int32_t n, d, f;
    int32_t tok;      // tokens of a tile, a multiple of 16
    int32_t rows;     // weight rows of a tile per CTA, a multiple of 8
    int32_t tiles_t, tiles_f;
    int32_t even;     // 1: every pair has an even share of all stages
    int32_t whole;    // in turn: tiles that are not split; they come first
    int32_t parts;    // in turn: units of each tile after them
    int32_t n_units;  // in turn: of all tiles; even shares: stages of all tiles
};

struct Unit {
    int f0, t0;    // first weight row of the pair's tile, first token
    int kb0, kb1;  // stages of the sum
    int parts;     // units of this tile
    int part;      // this one
    int split;     // number of this tile among those that may be split, where parts > 1
    int first;     // even shares: the pair that has the tile's first unit
};

__host__ __device__ inline int stages_of(const Schedule& p) { return (p.d + kKB - 1) / kKB; }

// First weight row and first token of a tile: groups of kGroupF row tiles, walked token
// tile by token tile.
__host__ __device__ inline void tile_at(const Schedule& p, int tile, Unit& r) {
    const int per = kGroupF * p.tiles_t;
    const int g = tile / per, rest = tile - g * per;
    const int rows = p.tiles_f - g * kGroupF < kGroupF ? p.tiles_f - g * kGroupF : kGroupF;
    const int t = rest / rows;
    r.t0 = t * p.tok;
    r.f0 = (g * kGroupF + (rest - t * rows)) * 2 * p.rows;
}

// The pair whose even share holds stage x of all.
__host__ __device__ inline int pair_of(const Schedule& p, int64_t x, int n_pairs) {
    return static_cast<int>((n_pairs * (x + 1) - 1) / p.n_units);
}

// The i-th unit of a pair; false where there is none.
__host__ __device__ inline bool unit_of(const Schedule& p, int pair, int n_pairs, int i, Unit& r) {
    const int n_kb = stages_of(p);
    if (p.even) {
        const int64_t from = static_cast<int64_t>(p.n_units) * pair / n_pairs;
        const int64_t to = static_cast<int64_t>(p.n_units) * (pair + 1) / n_pairs;
        const int64_t tile = from / n_kb + i, first = tile * n_kb;
        if (first >= to) return false;
        r.kb0 = from > first ? static_cast<int>(from - first) : 0;
        r.kb1 = to < first + n_kb ? static_cast<int>(to - first) : n_kb;
        r.first = pair_of(p, first, n_pairs);
        r.parts = pair_of(p, first + n_kb - 1, n_pairs) - r.first + 1;
        r.part = pair - r.first;
        r.split = static_cast<int>(tile);
        tile_at(p, static_cast<int>(tile), r);
        return true;
    }
    int u = pair + i * n_pairs;
    if (u >= p.n_units) return false;
    r.parts = 1;
    r.part = r.split = r.first = 0;
    if (u >= p.whole) {
        r.parts = p.parts;
        r.split = (u - p.whole) / p.parts;
        r.part = (u - p.whole) - r.split * p.parts;
        u = p.whole + r.split;
    }
    tile_at(p, u, r);
    r.kb0 = n_kb * r.part / r.parts;
    r.kb1 = n_kb * (r.part + 1) / r.parts;
    return true;
}

// Where the sums of unit k of a split tile are kept, of 2 * n_pairs places.
__host__ __device__ inline int piece_of(const Schedule& p, const Unit& un, int k, int n_pairs) {
    if (!p.even) return un.split * un.parts + k;
    const int pair = un.first + k;  // it has at most two parts of tiles: its first tile's and its last's
    const int64_t from = static_cast<int64_t>(p.n_units) * pair / n_pairs;
    return 2 * pair + (from / stages_of(p) == un.split ? 0 : 1);
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Pairs that a launch has, out of those that run at once.
inline int pairs_of(const Schedule& p, int pairs) { return p.n_units < pairs ? p.n_units : pairs; }

// Tiles and splits for n tokens.  In SM cycles, a stage costs what bounds it: the MMAs
// (4 a token), their issue and what it waits for (kIssue), or the weights' way from memory
// (16 bytes a row over 3 cycles at 24 bytes a cycle and SM).  A turn of units costs
// kTurn more; a tile in pieces kSplit for meeting, and 32 a token for each piece but one that
// the last pair there reads.
inline void plan(Schedule& p, int64_t pairs) {
    constexpr int64_t kIssue = 800, kTurn = 700, kSplit = 9000;
    const int64_t n_kb = ceil_div(p.d, kKB);
    p.tiles_t = static_cast<int32_t>(ceil_div(p.n, kMaxTok));
    p.tok = static_cast<int32_t>(ceil_div(ceil_div(p.n, p.tiles_t), 16) * 16);
    // rows are multiples of 8: 16 bytes of a row of results
    const int64_t most = p.f < 2 * kMaxRows ? ceil_div(p.f, 16) * 8 : kMaxRows;
    int64_t best = -1;
    const auto take = [&](int64_t cost, int64_t rows, int64_t tiles_f, bool even, int64_t whole, int64_t parts,
                          int64_t units) {
        if (best >= 0 && cost >= best) return;
        best = cost;
        p.rows = static_cast<int32_t>(rows);
        p.tiles_f = static_cast<int32_t>(tiles_f);
        p.even = even ? 1 : 0;
        p.whole = static_cast<int32_t>(whole);
        p.parts = static_cast<int32_t>(parts);
        p.n_units = static_cast<int32_t>(units);
    };
    for (int64_t wide = most; wide > 0; wide -= 8) {
        const int64_t tiles_f = ceil_div(p.f, 2 * wide), balanced = ceil_div(p.f, 16 * tiles_f) * 8;
        const int64_t rows = ceil_div(p.f, 2 * balanced) == tiles_f ? balanced : wide;  // the same rows in every tile
        const int64_t tiles = p.tiles_t * tiles_f;
        const int64_t turns = tiles / pairs, rest = tiles % pairs;
        int64_t stage = 4 * p.tok;
        if (stage < kIssue) stage = kIssue;
        if (stage < 16 * rows / 3) stage = 16 * rows / 3;
        for (int64_t s = 1; s <= kMaxParts && s <= n_kb && (s == 1 || rest * s <= pairs); ++s) {
            int64_t cost = turns * (n_kb * stage + kTurn);
            if (rest > 0) cost += ceil_div(n_kb, s) * stage + kTurn;
            if (s > 1) cost += kSplit + 32 * p.tok * (s - 1);
            const int64_t whole = s > 1 ? tiles - rest : tiles;
            take(cost, rows, tiles_f, false, whole, s, s > 1 ? whole + rest * s : tiles);
            if (rest == 0) break;
        }
        if (tiles <= pairs) {
            const int64_t share = ceil_div(tiles * n_kb, pairs);
            const int64_t parts = ceil_div(n_kb, share) + 1;
            take(share * stage + 2 * kTurn + kSplit + 32 * p.tok * (parts - 1), rows, tiles_f, true, 0, 1, tiles * n_kb);
        }
    }
}

}  // namespace i8
}  // namespace hk
