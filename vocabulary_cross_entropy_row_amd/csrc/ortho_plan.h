// Which tiles the products of an orthogonalised update take (host code alone, so that it can be looked at
// without a GPU; orthogonalise.hip has the tiles).
#pragma once

#include <algorithm>
#include <cmath>
#include <stdint.h>

namespace lce {
namespace ortho_plan {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

enum { BIG, MID, SMALL, MID_DEEP, FINE, SHAPES };   // FINE: fine_kernel
constexpr int kSide[SHAPES] = {256, 128, 64, 128, 32}, kPerCu[SHAPES] = {1, 2, 2, 1, 2};
// us of a step of 64 of K with one and two workgroups on a compute unit, and of a tile's start and end.
// Fitted to the times of all five steps over 221 random shapes (batches of 1 to 16, 65 to 16384 rows and
// columns, fp16's X alone in B X) with each shape for each product, replayed from a graph: off by 12% (root
// mean square), and the choice that the estimates make 2% slower than the fastest measured one on geometric
// average.
constexpr double kStepUs[SHAPES][2] = {{1.03, 0}, {0.65, 0.94}, {0.33, 0.33}, {0.45, 0}, {0.27, 0.57}};
constexpr double kTileUs[SHAPES] = {12.0, 3.4, 2.1, 4.3, 2.1};
constexpr double kEven = 1.94;   // a step where workgroups are at different places of K and share less in the caches
constexpr double kFoldUs = 3.0, kFoldRate = 10e6;   // the launch that adds pieces up, and its bytes a us
constexpr int kCus = 256;

struct Plan {
    int shape, groups;      // groups == total: a workgroup a tile
    int64_t tiles, total;   // of one matrix, of the batch
};
inline int64_t tiles_of(int64_t rows_x, int64_t rows_w, int side, bool sym) {
    const int64_t t = ceil_div(rows_x, side);
    return sym ? t * (t + 1) / 2 : t * ceil_div(rows_w, side);
}
// The shape with the least estimated time, a workgroup a tile; or, with `ranges` (X X^T, whose K is the longer
// side), as many workgroups as fit on the card, with equal ranges of all steps, which costs each two ends
// and the launch that adds the pieces up.  FINE is no faster for X X^T (K is not short: 256 x 1024 92 us, with
// tiles of 64 89) and is not built for it.
inline Plan plan_of(int64_t batch, int64_t rows_x, int64_t rows_w, int64_t steps, bool sym, bool ranges) {
    Plan best{SMALL, 0, 0, 0};
    double best_us = 1e30;
    for (int i = 0; i < SHAPES; ++i) {
        if (i == FINE && ranges) continue;
        const int64_t tiles = tiles_of(rows_x, rows_w, kSide[i], sym), total = batch * tiles, slots = static_cast<int64_t>(kCus) * kPerCu[i];
        double whole = static_cast<double>(total / slots) * (static_cast<double>(steps) * kStepUs[i][kPerCu[i] - 1] + kTileUs[i]);
        if (total % slots) whole += static_cast<double>(steps) * kStepUs[i][ceil_div(total % slots, kCus) - 1] + kTileUs[i];
        if (whole < best_us - 1e-9) {
            best_us = whole;
            best = {i, static_cast<int>(total), tiles, total};
        }
        const int64_t groups = std::min(slots, total * steps / 4);
        if (!ranges || groups == total || groups < 1) continue;
        const double depth = static_cast<double>(ceil_div(total * steps, groups)), pieces = static_cast<double>(std::min(2 * total, total + groups));
        const double even = depth * kStepUs[i][ceil_div(groups, kCus) - 1] * kEven + 2.0 * kTileUs[i] + kFoldUs +
                            pieces * kSide[i] * kSide[i] * 8 / kFoldRate;
        if (even < best_us - 1e-9) {
            best_us = even;
            best = {i, static_cast<int>(groups), tiles, total};
        }
    }
    return best;
}

// ---- what fp16 holds X and the off-diagonal parts of A and B times -------------------------------
//
// X = G / ||G|| has singular values up to 1, and p(s) = a s + b s^3 + c s^5 of them after a step.  With m the most
// that they can be, |X| <= m, |A| <= m^2 and |B| <= the largest |b t + c t^2| up to t = m^2, and so is every
// value of theirs: powers of two that leave these below 2^15 never overflow fp16.

// the largest |p(s)| for s from 0 to m: at m, or where p' is 0
inline double peak(double a, double b, double c, double m) {
    auto p = [&](double t) { return std::fabs(std::sqrt(t) * (a + t * (b + c * t))); };
    double top = p(m * m);
    auto at = [&](double t) {
        if (t > 0.0 && t < m * m) top = std::max(top, p(t));   // false of NaN
    };
    const double d = 9.0 * b * b - 20.0 * a * c;   // of a + 3 b t + 5 c t^2
    if (d >= 0.0) {
        const double q = -0.5 * (3.0 * b + std::copysign(std::sqrt(d), b));
        at(q / (5.0 * c));
        at(a / q);
    }
    return top;
}
// the largest |b t + c t^2| for t from 0 to u
inline double peak_b(double b, double c, double u) {
    double top = std::fabs(u * (b + c * u));
    const double t = -b / (2.0 * c);
    if (t > 0.0 && t < u) top = std::max(top, std::fabs(t * (b + c * t)));
    return top;
}
// Past a value of 256 the powers would leave small values of A few bits; terms past 2^100 leave fp32.
constexpr double kMaxValue = 256.0, kMaxTerm = 0x1p100;   // of X before a step; of a, b m^2 and c m^4

struct Powers {
    bool fit;          // nothing passes kMaxValue or kMaxTerm; the others mean nothing if not
    float x, o, b;
    bool rest;         // whether B X takes what fp16 leaves of X too
};
// The powers are at most 2^14, 2^10 and 2^8, which the default coefficients (m = 1.21) have.
//
// a X + B X is (a + B) X, whose rows stay in the space of X's, if both terms have the same X.  With fp16's X in
// the product alone, what fp16 leaves makes directions that X did not have, of the second order in fp16's
// step, and the steps multiply them by `a` each: about 9e-4 |a|^steps / r of the result (Frobenius norm) where G has
// one direction, as the definition with the kernel's roundings shows (five default steps: 64 x 64 5.4e-3, 512 x 1024
// 8.6e-4; eight: 1.4e-1, 2.2e-2).  Where that could reach half of the bf16 output's rounding, 1.7e-3, the product takes
// both (6.0e-4; eight: 2.1e-3, 2.7e-3, where products in fp32 give 1.7e-3, 2.6e-3), for twice its instructions.
// Up to 64 rows always: the kernel for them has one form.
inline Powers powers_of(int64_t r, int steps, double a, double b, double c) {
    double m = 1.0, x = 0.0, o = 0.0, p = 0.0;
    Powers s{true, 0, 0, 0, r <= 64};
    for (int k = 0; k < steps && s.fit; ++k) {
        x = std::max(x, m);
        o = std::max(o, m * m);
        p = std::max(p, peak_b(b, c, m * m));
        s.fit = m <= kMaxValue && std::fabs(a) <= kMaxTerm && std::fabs(b) * m * m <= kMaxTerm &&
                std::fabs(c) * m * m * m * m <= kMaxTerm;
        m = peak(a, b, c, m) * (1.0 + 0x1p-8);   // and what the roundings add
    }
    auto power = [](double v, int most) {
        return std::ldexp(1.0f, v > 0.0 ? static_cast<int>(std::min<double>(most, std::floor(15.0 - std::log2(v)))) : most);
    };
    s.x = power(x, 14);
    s.o = power(o, 10);
    s.b = power(p, 8);
    s.rest = s.rest || steps * std::log(std::fabs(a)) > std::log(static_cast<double>(r));
    return s;
}

}  // namespace ortho_plan
}  // namespace lce
