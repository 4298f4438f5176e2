// Checks csrc/gated_ff_schedule.cuh on the CPU.  For many sizes and numbers of
// pairs, and each launch of a call:
//   * every unit goes to one pair, before the pair's first "no more";
//   * every tile's boxes are summed once, by its units, in order, none empty;
//   * the tiles cover the result once and begin inside it;
//   * pieces and counts of split tiles are each unit's own and fit the workspace.
// With "n d f" arguments it prints how those sizes are split at 76 pairs instead:
// whole tiles, units of the tiles after them, units of a tile of dX.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <set>
#include <tuple>
#include <vector>

#include "gated_ff_schedule.cuh"

using namespace hk::ff;

namespace {

FfSchedule sizes(int n, int d, int f) {
    FfSchedule p{};
    p.n = n;
    p.d = d;
    p.f = f;
    return p;
}

#define CHECK(x)                                                                                             \
    do {                                                                                                     \
        if (!(x)) {                                                                                          \
            std::printf("%s: n %d d %d f %d pairs %d launch %d\n", #x, p.n, p.d, p.f, pairs, kWhat);         \
            return false;                                                                                    \
        }                                                                                                    \
    } while (0)

template <int kWhat>
bool covered(const FfSchedule& p, int pairs, bool want_x, bool want_w) {
    const int n_pairs = p.n_units < pairs ? p.n_units : pairs;
    std::vector<char> taken(p.n_units, 0);
    for (int pair = 0; pair < n_pairs; ++pair)
        for (int k = 0, u; (u = unit_of<kWhat>(p, pair, n_pairs, k)) >= 0; ++k) {
            CHECK(u < p.n_units && !taken[u]);
            taken[u] = 1;
        }
    for (int u = 0; u < p.n_units; ++u) CHECK(taken[u]);

    struct Tile {
        int next = 0, parts = 0, split = 0, n_kb = 0;
    };
    std::map<std::tuple<int, int, int, int>, Tile> tiles;
    std::set<int> pieces, counts;
    for (int u = 0; u < p.n_units; ++u) {
        const Unit un = unit_at<kWhat>(p, u);
        CHECK(un.kb0 < un.kb1);
        Tile& t = tiles[{un.kind, un.which, un.m0, un.n0}];
        if (un.part == 0) {
            CHECK(t.parts == 0);
            t.parts = un.parts;
            t.split = un.split;
            if (un.parts > 1) CHECK(un.split < pairs && counts.insert(un.split).second);
        }
        // units come in the order of their pieces
        CHECK(t.parts == un.parts && t.split == un.split && un.kb0 == t.next && un.part < un.parts);
        t.next = un.kb1;
        if (un.parts > 1) {
            const int piece = un.split * un.parts + un.part;
            CHECK(piece < pairs && pieces.insert(piece).second);
        }
        const int rows = un.kind == 2 ? p.f : p.n, cols = un.kind == 0 ? p.f : p.d;
        CHECK(un.m0 >= 0 && un.m0 < rows && un.n0 >= 0 && un.n0 < cols);
        CHECK(un.m0 % 256 == 0 && un.n0 % (un.kind == 0 ? 128 : 256) == 0);
        t.n_kb = un.kind == 0 ? (p.d + 63) / 64 : un.kind == 1 ? 2 * ((p.f + 63) / 64) : (p.n + 63) / 64;
        if (un.kind == 1) CHECK(un.half == (p.f + 63) / 64);
    }
    for (const auto& [key, t] : tiles) CHECK(t.next == t.n_kb);
    const int64_t x = int64_t((p.n + 255) / 256), f2 = (p.f + 255) / 256, d2 = (p.d + 255) / 256;
    CHECK(static_cast<int64_t>(tiles.size()) ==
          (kWhat == kGradients ? (want_x ? x * d2 : 0) + (want_w ? 2 * f2 * d2 : 0) : x * ((p.f + 127) / 128)));
    return true;
}

long split_forward = 0, split_after_whole = 0, split_x = 0, skips = 0;

bool check(int n, int d, int f, int pairs) {
    FfSchedule p = sizes(n, d, f);
    plan_projections(p, pairs);
    split_forward += p.parts > 1;
    split_after_whole += p.parts > 1 && p.whole > 0;
    if (!covered<kForward>(p, pairs, false, false)) return false;
    for (int want = 1; want < 4; ++want) {
        FfSchedule q = sizes(n, d, f);
        plan_gradients(q, pairs, want & 1, want & 2);
        split_x += q.parts > 1;
        skips += q.skip > 0;
        if (!covered<kGradients>(q, pairs, want & 1, want & 2)) return false;
    }
    return true;
}

}  // namespace

int main(int argc, char** argv) {
    if (argc > 1) {
        for (int i = 1; i + 2 < argc; i += 3) {
            FfSchedule p = sizes(std::atoi(argv[i]), std::atoi(argv[i + 1]), std::atoi(argv[i + 2])), q = p;
            plan_projections(p, 76);
            plan_gradients(q, 76, true, true);
            std::printf("%d %d %d\n", p.whole, p.parts, q.parts);
        }
        return 0;
    }
    std::mt19937 rng(3);
    const auto wide = [&](double lo, double hi) {  // even over the logarithm
        return static_cast<int>(lo * std::pow(hi / lo, std::uniform_real_distribution<double>(0, 1)(rng)));
    };
    for (int i = 0; i < 4000; ++i) {
        const int pairs = i % 3 == 0 ? wide(1, 100) : 76;
        if (!check(wide(1, 9000), 8 * wide(1, 1100), 8 * wide(1, 1400), pairs)) return 1;
    }
    for (int n : {1, 128, 129, 255, 256, 257, 4096, 8192})
        for (int d : {8, 64, 72, 4096, 65536})
            for (int f : {8, 128, 136, 11008}) {
                if (!check(n, d, f, 76)) return 1;
                if (d < 65536 && !check(n, f, d, 76)) return 1;
            }
    std::printf("schedule ok: split %ld, after whole tiles %ld, dX %ld, turns sat out %ld\n", split_forward,
                split_after_whole, split_x, skips);
    return split_forward > 500 && split_after_whole > 50 && split_x > 500 && skips > 500 ? 0 : 1;
}
