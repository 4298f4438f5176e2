// Checks csrc/int8_schedule.cuh on the CPU.  For many sizes and numbers of pairs:
//   * tiles are ones the MMA and the copies can take (tokens a multiple of 16, at most
//     192; a multiple of 8, at most 128, of weight rows per CTA), begin inside the result and cover it once;
//   * every tile's stages are summed once, by its units, in order, none empty;
//   * pieces and counts of split tiles are each unit's own and fit the workspace, and no pair has a
//     unit after one of a split tile.
// With "n d f" arguments it prints how those sizes are laid out at 76 pairs instead:
// tokens and rows of a tile, whole tiles, units of the tiles after them.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <set>
#include <utility>

#include "int8_schedule.cuh"

using namespace hk::i8;

namespace {

#define CHECK(x)                                                                              \
    do {                                                                                      \
        if (!(x)) {                                                                           \
            std::printf("%s: n %d d %d f %d pairs %d\n", #x, p.n, p.d, p.f, pairs);           \
            return false;                                                                     \
        }                                                                                     \
    } while (0)

long split = 0, split_after_whole = 0, low = 0;

bool check(int n, int d, int f, int pairs) {
    Schedule p{};
    p.n = n;
    p.d = d;
    p.f = f;
    plan(p, pairs);
    CHECK(p.tok % 16 == 0 && p.tok >= 16 && p.tok <= kMaxTok && p.rows % 8 == 0 && p.rows >= 8 && p.rows <= kMaxRows);
    CHECK(p.parts >= 1 && p.n_units >= 1 && p.whole >= 0);
    split += p.parts > 1;
    split_after_whole += p.parts > 1 && p.whole > 0;
    low += p.rows < kMaxRows;
    struct Tile {
        int next = 0, parts = 0, split = 0;
    };
    std::map<std::pair<int, int>, Tile> tiles;
    std::set<int> pieces, counts;
    const int n_kb = (d + kKB - 1) / kKB;
    for (int u = 0; u < p.n_units; ++u) {
        const Unit un = unit_at(p, u);
        CHECK(un.kb0 < un.kb1 && un.kb1 <= n_kb && un.part >= 0 && un.part < un.parts);
        CHECK(un.f0 >= 0 && un.f0 < f && un.t0 >= 0 && un.t0 < n);
        CHECK(un.f0 % (2 * p.rows) == 0 && un.t0 % p.tok == 0);
        Tile& t = tiles[{un.f0, un.t0}];
        if (un.part == 0) {
            CHECK(t.parts == 0);
            t.parts = un.parts;
            t.split = un.split;
            if (un.parts > 1) CHECK(un.split < pairs && counts.insert(un.split).second);
        }
        CHECK(t.parts == un.parts && t.split == un.split && un.kb0 == t.next);
        t.next = un.kb1;
        if (un.parts > 1) {
            const int piece = un.split * un.parts + un.part;
            CHECK(piece < pairs && pieces.insert(piece).second);
            CHECK(u + pairs >= p.n_units);  // the last unit of its pair
        }
    }
    for (const auto& [key, t] : tiles) CHECK(t.next == n_kb);
    CHECK(static_cast<int64_t>(tiles.size()) ==
          int64_t((f + 2 * p.rows - 1) / (2 * p.rows)) * ((n + p.tok - 1) / p.tok));
    return true;
}

}  // namespace

int main(int argc, char** argv) {
    if (argc > 1) {
        for (int i = 1; i + 2 < argc; i += 3) {
            Schedule p{};
            p.n = std::atoi(argv[i]);
            p.d = std::atoi(argv[i + 1]);
            p.f = std::atoi(argv[i + 2]);
            plan(p, 76);
            std::printf("%d %d %d %d\n", p.tok, p.rows, p.whole, p.parts);
        }
        return 0;
    }
    std::mt19937 rng(5);
    const auto wide = [&](double lo, double hi) {  // even over the logarithm
        return static_cast<int>(lo * std::pow(hi / lo, std::uniform_real_distribution<double>(0, 1)(rng)));
    };
    for (int i = 0; i < 6000; ++i) {
        const int pairs = i % 3 == 0 ? wide(1, 100) : 76;
        if (!check(wide(1, 9000), 16 * wide(1, 700), 8 * wide(1, 1400), pairs)) return 1;
    }
    for (int n : {1, 16, 17, 192, 193, 385, 8192, 1 << 20})
        for (int d : {16, 128, 144, 4096, 65536})
            for (int f : {8, 128, 136, 11008, 65536})
                if (!check(n, d, f, 76)) return 1;
    std::printf("schedule ok: split %ld, after whole tiles %ld, fewer rows %ld\n", split, split_after_whole, low);
    return split > 500 && split_after_whole > 50 && low > 1000 ? 0 : 1;
}
