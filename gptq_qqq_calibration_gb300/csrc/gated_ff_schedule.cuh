// Who computes what in the feed-forward kernels of SM pairs: the tiles of each
// contraction, the units a tile is split in, and the pair that takes each unit.
// Host and device functions, so that the kernels, the host library and a CPU test
// of the schedule (tests/ff_schedule_check.cu) run the same code.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace hk {
namespace ff {

constexpr int kKB = 64;     // contraction steps of one stage: a box
constexpr int kGroupM = 8;  // row tiles that run side by side (their B boxes meet in L2)

enum { kForward, kActGrad, kGradients };  // what a launch computes

struct FfSchedule {
    int32_t n, d, f;
    int32_t whole;    // kForward, kActGrad: tiles that are not split; they come first
    int32_t parts;    // units of each tile after them, or of each tile of dX
    int32_t units_x;  // kGradients: units of dX (first), then 2 * tiles_w tiles of dWg and dWu
    int32_t tiles_w;
    int32_t n_units;
    int32_t skip;     // kGradients: turns of dW tiles that one tile of dX is worth
};

// Tile u of tm x tn, in groups of kGroupM row tiles walked column by column.
__host__ __device__ inline void tile_at(int u, int tm, int tn, int& m, int& n) {
    const int per = kGroupM * tn;
    const int g = u / per, r = u - g * per;
    const int rows = tm - g * kGroupM < kGroupM ? tm - g * kGroupM : kGroupM;
    n = r / rows;
    m = g * kGroupM + (r - n * rows);
}

// The k-th unit of a pair, or -1.  Units go to the pairs in turn.  The tiles of
// dX are long (their sums run over f twice), so some pairs have one more of them
// than the others; those sit out the first p.skip turns of the tiles of dW.
template <int kWhat>
__host__ __device__ inline int unit_of(const FfSchedule& p, int pair, int n_pairs, int k) {
    int u = pair + k * n_pairs;
    if constexpr (kWhat == kGradients) {
        if (u >= p.units_x) {
            const int more = p.units_x % n_pairs, mine = p.units_x / n_pairs + (pair < more ? 1 : 0);
            const int turn = k - mine + (pair < more ? p.skip : 0);
            u = p.units_x + (turn < p.skip ? turn * (n_pairs - more) + pair - more
                                           : p.skip * (n_pairs - more) + (turn - p.skip) * n_pairs + pair);
        }
    }
    return u < p.n_units ? u : -1;
}

struct Unit {
    int kind;   // 0: X times weights, 1: dX, 2: dW
    int m0, n0;  // first row of A and of B (kind 0: of each weight)
    int which;  // kind 2: 0 = gate, 1 = up
    int kb0, kb1;  // boxes of the sum
    int half;   // kind 1: boxes of the gate half of the sum
    int parts;  // units of this tile
    int part;   // this one
    int split;  // split tiles before this one
};

template <int kWhat>
__host__ __device__ inline Unit unit_at(const FfSchedule& p, int u) {
    Unit r{};
    int m, n, n_kb;
    r.parts = 1;
    if constexpr (kWhat != kGradients) {
        if (u >= p.whole) {
            r.parts = p.parts;
            r.split = (u - p.whole) / p.parts;
            r.part = (u - p.whole) - r.split * p.parts;
            u = p.whole + r.split;
        }
        tile_at(u, (p.n + 255) / 256, (p.f + 127) / 128, m, n);
        r.m0 = m * 256;
        r.n0 = n * 128;
        n_kb = (p.d + kKB - 1) / kKB;
    } else if (u < p.units_x) {
        r.parts = p.parts;
        r.split = u / p.parts;
        r.part = u - r.split * p.parts;
        tile_at(r.split, (p.n + 255) / 256, (p.d + 255) / 256, m, n);
        r.kind = 1;
        r.m0 = m * 256;
        r.n0 = n * 256;
        r.half = (p.f + kKB - 1) / kKB;
        n_kb = 2 * r.half;
    } else {
        u -= p.units_x;
        r.which = u >= p.tiles_w ? 1 : 0;
        tile_at(u - r.which * p.tiles_w, (p.f + 255) / 256, (p.d + 255) / 256, m, n);
        r.kind = 2;
        r.m0 = m * 256;
        r.n0 = n * 256;
        n_kb = (p.n + kKB - 1) / kKB;
    }
    r.kb0 = n_kb * r.part / r.parts;
    r.kb1 = n_kb * (r.part + 1) / r.parts;
    return r;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Units to split a tile of n_kb boxes in, when `tiles` of them run side by side
// and the pairs have `share` boxes of work each in all.  A box takes 512 cycles at
// the tensor cores' rate; a split costs about as much as 8 boxes for the pieces'
// way to memory and the pairs' meeting, and 4 for reading each piece again.  It
// has to promise a fourteenth of the time (129 tokens at 4,096 x 11,008, backward:
// 163 us unsplit, 129 with dX in 2, 145 in 3; 1,024 at 2,048 x 5,632: 94 unsplit,
// 102 in 2; 203 at 520 x 1,400: 30.4 unsplit, 27.2 in 3).
inline int32_t parts_of(int64_t tiles, int64_t n_kb, int64_t pairs, int64_t share) {
    const auto cost = [&](int64_t s) {
        const int64_t longest = ceil_div(n_kb, s);
        return (longest > share ? longest : share) + (s > 1 ? 8 + 4 * s : 0);
    };
    int64_t best = 1;
    for (int64_t s = 2; s <= 8 && tiles * s <= pairs; ++s)
        if (14 * cost(s) < 13 * cost(1) && cost(s) < cost(best)) best = s;
    return static_cast<int32_t>(best);
}

// Units of X times the weights: whole rounds of tiles, then the rest, split.
inline void plan_projections(FfSchedule& p, int64_t pairs) {
    const int64_t tiles = ceil_div(p.n, 256) * ceil_div(p.f, 128), rest = tiles % pairs;
    p.parts = rest > 0 ? parts_of(rest, ceil_div(p.d, kKB), pairs, 0) : 1;
    p.whole = static_cast<int32_t>(p.parts > 1 ? tiles - rest : tiles);
    p.n_units = static_cast<int32_t>(p.parts > 1 ? p.whole + rest * p.parts : tiles);
}

// Units of dX, and of both weight gradients.
inline void plan_gradients(FfSchedule& p, int64_t pairs, bool want_x, bool want_w) {
    const int64_t tiles_x = want_x ? ceil_div(p.n, 256) * ceil_div(p.d, 256) : 0;
    const int64_t tiles_w = want_w ? ceil_div(p.f, 256) * ceil_div(p.d, 256) : 0;
    const int64_t kb_x = 2 * ceil_div(p.f, kKB), kb_w = ceil_div(p.n, kKB);
    // in the share of each pair a tile of dW counts at least its write-out, some 10 boxes
    p.parts = parts_of(tiles_x, kb_x, pairs,
                       ceil_div(tiles_x * kb_x + 2 * tiles_w * (kb_w > 10 ? kb_w : 10), pairs));
    p.units_x = static_cast<int32_t>(tiles_x * p.parts);
    p.tiles_w = static_cast<int32_t>(tiles_w);
    p.n_units = p.units_x + 2 * p.tiles_w;
    const int64_t kb_unit = kb_x / p.parts;
    p.skip = want_x && want_w ? static_cast<int32_t>((kb_unit + kb_w / 2) / kb_w) : 0;
}

}  // namespace ff
}  // namespace hk
