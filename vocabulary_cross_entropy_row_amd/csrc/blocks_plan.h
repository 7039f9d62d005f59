// Which tiles and K splits the product with a scale for each block of 128 takes (host code alone, so that it
// can be looked at without a GPU; linear_blocks.hip has the tiles).
#pragma once

#include "linear_plan.h"

namespace lce {
namespace blocks_plan {

using linear_plan::BIG;
using linear_plan::ceil_div;
using linear_plan::Cost;
using linear_plan::kCus;
using linear_plan::kMaxSplits;
using linear_plan::kMaxThreads;
using linear_plan::LOW;
using linear_plan::Plan;
using linear_plan::round_up;
using linear_plan::ROWS16;
using linear_plan::ROWS32;
using linear_plan::SHAPES;
using linear_plan::TINY;
using linear_plan::WIDE;

// The terms are linear_plan.h's.  Fitted to the times of each shape, with 1 to 16 splits, over 500 random
// products (n 1 to 8192, K 128 to 16384, M 64 to 202048) with each kind of scales, replayed from a graph:
// off by 9 to 11% on those (root mean square; 16 to 22% with the tiles of 16 and 32 tokens), and the choice
// that the estimates make 2% slower than the fastest measured one on geometric average.
struct ShapeInfo {
    int bf, bt, per_cu, threads;
    Cost pow2, any;   // e8m0 scales on both sides, and others
};
constexpr ShapeInfo kShapes[SHAPES] = {
    {256, 256, 1, 512, {{1.20, 0, 0}, 7.3, 2.4, 3.8e6, 1.1, 6.3e6}, {{1.43, 0, 0}, 7.5, 2.4, 3.6e6, 1.4, 6.4e6}},
    {256, 128, 1, 512, {{0.75, 0, 0}, 5.8, 1.5, 4.6e6, 1.5, 6.2e6}, {{0.91, 0, 0}, 5.8, 1.6, 4.4e6, 1.5, 6.2e6}},
    {128, 64, 2, 256, {{0.38, 0.76, 0}, 3.0, 1.4, 5.2e6, 2.4, 5.8e6}, {{0.52, 0.83, 0}, 3.2, 1.4, 5.2e6, 2.4, 6.1e6}},
    {64, 32, 3, 128, {{0.36, 0.50, 0.53}, 2.8, 1.1, 5.1e6, 2.3, 5.0e6}, {{0.39, 0.52, 0.53}, 2.9, 1.2, 5.0e6, 2.2, 5.0e6}},
    {16, 16, 2, 512, {{0.08, 0.24, 0}, 4.0, 0.0, 3.5e6, 0, 1}, {{0.06, 0.22, 0}, 4.9, 0.0, 3.4e6, 0, 1}},
    {16, 32, 3, 512, {{0.15, 0.36, 0.55}, 4.1, 0.0, 4.0e6, 0, 1}, {{0.14, 0.35, 0.55}, 4.7, 0.0, 4.0e6, 0, 1}},
};

inline Plan plan_of(int64_t n, int64_t K, int64_t M, bool pow2) {
    const int64_t steps = std::max<int64_t>(1, ceil_div(K, 128));
    const double bytes = static_cast<double>(n + M) * K + 2.0 * n * M;
    Plan best{BIG, 1};
    double best_us = 1e30;
    for (int i = 0; i < SHAPES; ++i) {
        const bool rows = i == ROWS16 || i == ROWS32;
        if (rows && (n > kShapes[i].bt || (i == ROWS32 && n <= kShapes[ROWS16].bt))) continue;
        const ShapeInfo &s = kShapes[i];
        const Cost &c = pow2 ? s.pow2 : s.any;
        const int64_t tiles = ceil_div(M, s.bf) * ceil_div(n, s.bt), slots = static_cast<int64_t>(kCus) * s.per_cu;
        for (int sp = 1; sp <= (rows ? 1 : kMaxSplits) && (sp == 1 || steps / sp >= 3); ++sp) {
            const double depth = static_cast<double>(ceil_div(steps, sp));
            const int64_t groups = tiles * sp, last = groups % slots;
            if (round_up(groups, 8) * s.threads > kMaxThreads) break;
            double us = static_cast<double>(groups / slots) * (depth * c.step[s.per_cu - 1] + c.tile);
            if (last) us += depth * c.step[ceil_div(last, kCus) - 1] + c.tile;
            us = std::max(us, bytes / c.rate) + c.launch;
            if (sp > 1) us += c.fold + 8.0 * sp * static_cast<double>(n) * round_up(M, 8) / c.fold_rate;
            if (us < best_us - 1e-9) {
                best_us = us;
                best = {i, sp};
            }
        }
    }
    return best;
}

}  // namespace blocks_plan
}  // namespace lce
