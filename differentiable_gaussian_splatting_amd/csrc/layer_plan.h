// layer_plan.h -- how the layers' matrix products are cut into tiles and splits
// of k, by the measured cost of a step.  Plain C++: nothing here needs a GPU.
#pragma once

#include <algorithm>
#include <cstdint>

namespace gsm {

// The tiles of a product.  kTiny is for operands with fewer than 8 values side
// by side (Stage in mm.h).
enum { kLarge = 0, kMedium = 1, kSmall = 2, kTiny = 3 };

// What n tiles on each compute unit take for one step of k: once us for
// every round of `resident` blocks and each us for every tile (measured, with
// one to eight tiles a unit: 128 x 128 x 64 through registers 1.0, 1.45 and 2.25
// us for one, two and three, 64 x 64 x 64 0.72, 1.2 and 2.2 for two, four and
// eight, 256 x 256 x 64 2.4 for one, loaded directly 2.15).
struct TileCost {
    int32_t m, n, k, resident;   // m x n results, steps of k
    double once, each;
};
constexpr TileCost kCost16[] = {{256, 256, 64, 1, 0.1, 2.3}, {128, 128, 64, 2, 0.5, 0.48}, {64, 64, 64, 5, 0.2, 0.25},
                                {64, 64, 64, 3, 0.3, 0.3}};
constexpr TileCost kCostDirect[] = {{256, 256, 64, 1, 0.1, 2.1}, {128, 128, 64, 2, 0.3, 0.46}, {64, 64, 64, 5, 0.2, 0.25},
                                    {64, 64, 64, 3, 0.3, 0.3}};
constexpr TileCost kCost32[] = {{256, 128, 32, 1, 0.1, 2.5}, {128, 128, 32, 2, 0.5, 1.35}, {64, 64, 32, 3, 0.3, 0.48},
                                {64, 64, 32, 3, 0.4, 0.5}};
constexpr double kJoinUs = 4.0;          // a further launch
constexpr double kJoinRate = 4e6;        // bytes per us of sums written and read

struct ProductShape {
    int64_t m, n, k;             // rows and columns of out
    bool a_col, b_col, gated;    // operands whose k runs down the columns; gated: 2 n columns of products
};

struct TilePlan {
    int64_t tm, tn;              // tiles
    int64_t full;                // the first `full` tiles are formed whole, the others in
    int32_t splits, tile;        // `splits` ranges of kper values of k,
    int64_t kper;                // a multiple of the tile's step,
    int64_t floats;              // whose sums take this much workspace
};

inline int64_t pieces(int64_t n, int64_t each) { return (n + each - 1) / each; }

// What `tiles` tiles cost in s ranges of k.
inline double tiles_us(int num_cu, const TileCost& c, int64_t tiles, int64_t steps, int64_t s)
{
    const int64_t blocks = tiles * s;
    const double step = pieces(blocks, (int64_t)c.resident * num_cu) * c.once + pieces(blocks, num_cu) * c.each;
    return (double)(pieces(steps, s) + 1) * step + (s > 1 ? kJoinUs + 8.0 * blocks * c.m * c.n / kJoinRate : 0.0);
}

// The tile and the tiles that are split, as the costs above make fastest.  Whole
// rounds of the card are formed whole; a last round that would leave most of
// it idle, or the only one, is split over k (8191 x 4097 over 2049 f16: 544
// tiles of 256 x 256 on 256 units).
inline TilePlan plan_tiles(int num_cu, bool f32, bool direct, const ProductShape& g)
{
    const int64_t n = g.n * (g.gated ? 2 : 1);
    const bool tiny = (!g.a_col && g.k < 8) || (g.a_col && g.m < 8) || (!g.b_col && g.k < 8) || (g.b_col && g.n < 8);
    const TileCost* costs = f32 ? kCost32 : direct ? kCostDirect : kCost16;
    TilePlan p{};
    double best = 0.0;
    int64_t best_s = 1;
    for (int t = tiny ? kTiny : kLarge; t <= (tiny ? kTiny : kSmall); ++t) {
        const TileCost& c = costs[t];
        const int64_t tiles = pieces(g.m, c.m) * pieces(n, c.n), steps = std::max<int64_t>(1, pieces(g.k, c.k));
        const int64_t slots = (int64_t)c.resident * num_cu;
        const double whole = tiles_us(num_cu, c, tiles, steps, 1);
        if (best == 0.0 || whole < best) {
            best = whole;
            best_s = 1;
            p.tile = t;
            p.full = tiles;
        }
        const int64_t rest = tiles % slots, full = tiles - rest;
        for (int64_t s = 2; rest > 0 && s <= steps && rest * s <= 2 * slots; s += std::max<int64_t>(1, s / 4)) {
            const double us = (full ? tiles_us(num_cu, c, full, steps, 1) : 0.0) + tiles_us(num_cu, c, rest, steps, s);
            if (us >= best) continue;
            best = us;
            best_s = s;
            p.tile = t;
            p.full = full;
        }
    }
    const TileCost& c = costs[p.tile];
    p.tm = pieces(g.m, c.m);
    p.tn = pieces(n, c.n);
    p.kper = pieces(std::max<int64_t>(1, pieces(g.k, c.k)), best_s) * c.k;
    p.splits = (int32_t)std::max<int64_t>(1, pieces(g.k, p.kper));
    if (p.splits == 1) p.full = p.tm * p.tn;
    p.floats = p.splits > 1 ? p.splits * (p.tm * p.tn - p.full) * c.m * c.n : 0;
    return p;
}

}  // namespace gsm
