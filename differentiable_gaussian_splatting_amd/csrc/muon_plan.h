// muon_plan.h -- tiles, padding and splits of the products of Muon's larger
// matrices, by the measured cost of a step.  Plain C++: nothing here needs a GPU.
#pragma once

#include <algorithm>
#include <cstdint>

#ifdef __HIPCC__
#define GS_BOTH __host__ __device__
#else
#define GS_BOTH
#endif

namespace gsm {

GS_BOTH constexpr int64_t padded(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// the products of a Newton-Schulz step
enum { kGram, kPoly, kNext };

// What a group's product takes with a tile: for a step of 32 values of k,
// once us for every round of `resident` tiles on each compute unit and each us
// for every tile (measured: 128 x 128 takes 1.3 and 2.0 us for one and two a
// unit, 64 x 64 0.9, 1.5 and 3.1 for two, four and eight, 256 x 256 3.1).
struct NewtonCost {
    int b, resident;
    double once, each;
};
constexpr NewtonCost kNewtonCosts[3] = {{256, 1, 0.1, 3.0}, {128, 2, 0.5, 0.75}, {64, 4, 0.2, 0.33}};

// tiles of a matrix's product, of its padded sides
template <int KIND, typename M>
int64_t tiles_of(const M& t, int64_t unit, int b)
{
    const int64_t rows = padded(t.rows, unit) / b, cols = padded(t.cols, unit) / b, s = std::min(rows, cols);
    return KIND == kNext ? rows * cols : s * (s + 1) / 2;
}

// J: a group of matrices, job.t[k].rows and .cols for k < job.count
template <int KIND, typename J>
double newton_us(int num_cu, const J& job, int64_t unit, int splits, const NewtonCost& c)
{
    const auto pieces = [](int64_t n, int64_t each) { return (n + each - 1) / each; };
    double work = 0.0, longest = 0.0;
    int64_t tiles = 0;
    for (int32_t k = 0; k < job.count; ++k) {
        const auto& t = job.t[k];
        const double steps = (double)pieces(KIND == kGram ? std::max(t.rows, t.cols) : std::min(t.rows, t.cols), 32 * splits) + 2.0;
        const int64_t n = tiles_of<KIND>(t, unit, c.b) * splits;
        tiles += n;
        work += (double)n * steps;
        longest = std::max(longest, steps);
    }
    const int64_t rounds = pieces(tiles, (int64_t)c.resident * num_cu), on_each = pieces(tiles, num_cu);
    return std::max(work / (double)tiles * ((double)rounds * c.once + (double)on_each * c.each), longest * (c.once + c.each));
}

// the cheapest tile of those that the unit is a multiple of, and its cost
template <int KIND, typename J>
int choose_tile(int num_cu, const J& job, int64_t unit, int splits, double* us)
{
    int best = 2;
    *us = newton_us<KIND>(num_cu, job, unit, splits, kNewtonCosts[2]);
    for (int k = 1; k >= 0 && unit % kNewtonCosts[k].b == 0; --k) {
        const double c = newton_us<KIND>(num_cu, job, unit, splits, kNewtonCosts[k]);
        if (c >= *us) continue;
        *us = c;
        best = k;
    }
    return best;
}

// The unit to which a group's sides are padded (the largest tile it may use),
// and how often G's product is split over its long k (few tiles, a few
// matrices of one long side each, leave the card idle otherwise).
template <typename J>
void choose_sizes(int num_cu, const J& job, int32_t* best_unit, int* best_splits)
{
    double least = 0.0;
    for (int unit = 64; unit <= 256; unit *= 2) {
        double poly, next, gram;
        choose_tile<kPoly>(num_cu, job, unit, 1, &poly);
        choose_tile<kNext>(num_cu, job, unit, 1, &next);
        int64_t s = 0;
        for (int32_t k = 0; k < job.count; ++k) {
            const int64_t side = padded(std::min(job.t[k].rows, job.t[k].cols), unit);
            s += side * side;
        }
        for (int splits = 1; splits <= 32; splits *= 2) {
            if (splits > 1 && splits * s > (1ll << 26)) break;
            choose_tile<kGram>(num_cu, job, unit, splits, &gram);
            if (splits > 1) gram += 5.0 + 4.0 * (splits + 1) * s / 3e6;   // the sums' launch and bytes
            const double us = gram + poly + next;
            if (least > 0.0 && us >= least) continue;
            least = us;
            *best_unit = unit;
            *best_splits = splits;
        }
    }
}

}  // namespace gsm
