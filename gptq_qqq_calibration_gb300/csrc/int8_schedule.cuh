// Who computes what in the 8-bit integer product on SM pairs: the tiles of
// Y^T = Wq Xq^T, the units a tile's sum is split in, and the pair that takes each.
// Host and device functions, so that the kernel, the host library and a CPU test of
// the schedule (tests/int8_schedule_check.cu) run the same code.
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
    int32_t whole;    // tiles that are not split; they come first
    int32_t parts;    // units of each tile after them
    int32_t n_units;
};

struct Unit {
    int f0, t0;    // first weight row of the pair's tile, first token
    int kb0, kb1;  // stages of the sum
    int parts, part, split;  // units of this tile, this one, split tiles before it
};

// Tiles run in groups of kGroupF row tiles, walked token tile by token tile.
__host__ __device__ inline Unit unit_at(const Schedule& p, int u) {
    Unit r{};
    r.parts = 1;
    if (u >= p.whole) {
        r.parts = p.parts;
        r.split = (u - p.whole) / p.parts;
        r.part = (u - p.whole) - r.split * p.parts;
        u = p.whole + r.split;
    }
    const int per = kGroupF * p.tiles_t;
    const int g = u / per, rest = u - g * per;
    const int rows = p.tiles_f - g * kGroupF < kGroupF ? p.tiles_f - g * kGroupF : kGroupF;
    const int t = rest / rows;
    r.t0 = t * p.tok;
    r.f0 = (g * kGroupF + (rest - t * rows)) * 2 * p.rows;
    const int n_kb = (p.d + kKB - 1) / kKB;
    r.kb0 = n_kb * r.part / r.parts;
    r.kb1 = n_kb * (r.part + 1) / r.parts;
    return r;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles and splits for n tokens.  In SM cycles, a stage costs what bounds it: the MMAs
// (4 a token), their issue and what it waits for (kIssue; kAlone less where no converter
// shares the MMAs' scheduler), or the weights' way from memory (16 bytes a row over 3 cycles
// at 24 bytes a cycle and SM).  A turn of units costs kTurn more.  Tiles in pieces cost their
// meeting, and the last pair's reading of each piece but its own: 10,000 cycles and 24 a token,
// or 5,000 and 12 where whole tiles come before them, whose way out it hides behind.  (Fitted:
// 1,000 tokens at 8,192 x 4,096 54.8 us, whole tiles alone 63.1; at 4,096 x 4,096 36.3 and 37.9; 37
// at 11,008 x 4,096 18.4 and 30.4; 200 at 4,096 x 4,096 17.3 us whole, 18.8 in pieces.)
inline void plan(Schedule& p, int64_t pairs) {
    constexpr int64_t kIssue = 800, kAlone = 100, kTurn = 700;
    const int64_t n_kb = ceil_div(p.d, kKB);
    p.tiles_t = static_cast<int32_t>(ceil_div(p.n, kMaxTok));
    p.tok = static_cast<int32_t>(ceil_div(ceil_div(p.n, p.tiles_t), 16) * 16);
    // rows are multiples of 8: 16 bytes of a row of results
    const int64_t most = p.f < 2 * kMaxRows ? ceil_div(p.f, 16) * 8 : kMaxRows;
    int64_t best = -1;
    for (int64_t wide = most; wide > 0; wide -= 8) {
        const int64_t tiles_f = ceil_div(p.f, 2 * wide), balanced = ceil_div(p.f, 16 * tiles_f) * 8;
        const int64_t rows = ceil_div(p.f, 2 * balanced) == tiles_f ? balanced : wide;  // the same rows in every tile
        const int64_t tiles = p.tiles_t * tiles_f;
        const int64_t turns = tiles / pairs, rest = tiles % pairs;
        int64_t stage = 4 * p.tok;
        if (stage < kIssue) stage = rows > 96 ? kIssue : kIssue - kAlone;
        if (stage < 16 * rows / 3) stage = 16 * rows / 3;
        for (int64_t s = 1; s <= kMaxParts && s <= n_kb && (s == 1 || rest * s <= pairs); ++s) {
            int64_t cost = turns * (n_kb * stage + kTurn);
            if (rest > 0) cost += ceil_div(n_kb, s) * stage + kTurn;
            if (s > 1) cost += turns > 0 ? 5000 + 12 * p.tok * (s - 1) : 10000 + 24 * p.tok * (s - 1);
            if (best < 0 || cost < best) {
                best = cost;
                p.rows = static_cast<int32_t>(rows);
                p.tiles_f = static_cast<int32_t>(tiles_f);
                p.whole = static_cast<int32_t>(s > 1 ? tiles - rest : tiles);
                p.parts = static_cast<int32_t>(s);
                p.n_units = static_cast<int32_t>(s > 1 ? p.whole + rest * s : tiles);
            }
            if (rest == 0) break;
        }
    }
}

}  // namespace i8
}  // namespace hk
