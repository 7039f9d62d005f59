// Which tiles and K splits the matrix product takes (host code alone, so that it can be looked at without
// a GPU; linear.hip has the tiles).
#pragma once

#include <stdint.h>

#include <algorithm>

namespace lce {
namespace linear_plan {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

enum { BIG, WIDE, LOW, TINY, ROWS16, ROWS32, SHAPES };   // ROWS: linear_rows_kernel, up to 16 and 32 tokens

// What a shape's workgroups cost, in us: a step of K with 1, 2 or 3 of them on a compute unit, a
// workgroup's start and end, the launch, and what its tile moves at (bytes per us); for a product split
// along K the second launch and the rate of the partial sums.  Fitted to the times of each shape, with
// 1 to 16 splits, over 208 random bf16 products (n 1 to 4096, K 256 to 8192, M 256 to 202048) and 112
// e4m3 ones, before outputs above 256 MB were streamed: on those products off by 10 to 14% (root mean
// square), and the choice that the estimates make 3% slower than the fastest measured one on geometric
// average.  They have not been held against other products.
struct Cost {
    double step[3], tile, launch, rate, fold, fold_rate;
};
struct ShapeInfo {
    int bf, bt, per_cu, threads;
    Cost bf16, e4m3;
};
constexpr ShapeInfo kShapes[SHAPES] = {
    {256, 256, 1, 512, {{1.22, 0, 0}, 7.5, 0.3, 4.0e6, 2.2, 5.5e6}, {{1.48, 0, 0}, 8.4, 0.8, 2.8e6, 1.1, 4.9e6}},
    {256, 128, 1, 512, {{0.82, 0, 0}, 5.5, 0.0, 4.3e6, 3.1, 6.1e6}, {{0.86, 0, 0}, 6.2, 0.2, 3.4e6, 2.7, 4.9e6}},
    {128, 64, 2, 256, {{0.38, 0.85, 0}, 0.1, 4.3, 4.8e6, 3.2, 6.4e6}, {{0.33, 0.89, 0}, 1.8, 3.2, 4.1e6, 3.1, 4.6e6}},
    {64, 32, 3, 128, {{0.28, 0.38, 0.58}, 0.4, 3.9, 4.7e6, 2.9, 4.8e6}, {{0.23, 0.51, 0.55}, 1.7, 2.6, 4.3e6, 3.0, 4.0e6}},
    {16, 16, 2, 512, {{0.04, 0.16, 0}, 4.7, 0.7, 4.0e6, 0, 1}, {{0.03, 0.19, 0}, 4.3, 1.1, 8.0e6, 0, 1}},
    {16, 32, 3, 512, {{0.10, 0.30, 0.55}, 2.4, 2.8, 8.0e6, 0, 1}, {{0.11, 0.24, 0.56}, 4.5, 0.0, 8.0e6, 0, 1}},
};
constexpr int kCus = 256;        // compute units of an MI355X
constexpr int kMaxSplits = 16;
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;   // of a launch

struct Plan {
    int shape, splits;
};
// The tile shape and K splits with the least estimated time: whole rounds of workgroups over the
// compute units, the last one as full as it is, and not less than the bytes take.
inline Plan plan_of(int64_t n, int64_t K, int64_t M, bool fp8) {
    const int es = fp8 ? 1 : 2;
    const int64_t steps = std::max<int64_t>(1, ceil_div(K * es, 128));
    const double bytes = static_cast<double>(n + M) * K * es + 2.0 * n * M;
    Plan best{BIG, 1};
    double best_us = 1e30;
    for (int i = 0; i < SHAPES; ++i) {
        const bool rows = i == ROWS16 || i == ROWS32;
        if (rows && (n > kShapes[i].bt || (i == ROWS32 && n <= kShapes[ROWS16].bt))) continue;
        const ShapeInfo &s = kShapes[i];
        const Cost &c = fp8 ? s.e4m3 : s.bf16;
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

}  // namespace linear_plan
}  // namespace lce
