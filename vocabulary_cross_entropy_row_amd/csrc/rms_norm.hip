// Root-mean-square norm with the residual's addition, forward and backward, for
// gfx950.
//
//   s    = x + residual, rounded to the stream's type (what the next layer reads)
//   rstd = 1 / sqrt(mean(s^2) + eps)
//   y    = s rstd (w + offset)                in the stream's type, or
//   q    = e4m3(y / scale), scale = max|y| / 448, one scale per row
//
// and with g = dL/dy, gs = dL/ds (from the stream's later readers), a = g (w + offset):
//
//   dL/dx = dL/dresidual = rstd (a - s rstd^2 mean(a s)) + gs
//   dL/dw = sum over rows of g s rstd
//
// Both are bound by memory: every value is read once and written once, so a row
// lives in the registers of LPR lanes (16 to 1024) between its load and its
// stores, K accesses of 16 bytes (E values) per lane.  gfx950 takes those at any
// address; only an access that reaches past the row's end goes value by value.
// 8192 x 6656 bf16 with a residual: forward 73 to 78 us (5.6 to 6.0 TB/s), backward
// 92 to 98 us (4.5 to 4.7 TB/s) and 5 us for the partial rows of dL/dw; 4096 x 8192 to
// 8 bits 42 to 44 us (5.3 to 5.6 TB/s).  A large copy reaches 4.9 TB/s.  Rows off the
// 16-byte boundaries cost more (a row stride of 6657: 91 and 119 us), and so does a cut
// last access, in bf16 most of all: 8192 x 6655 in rows of 6656 105 and 266 us, packed
// 123 and 294; fp32 157 and 183, 150 and 164 at 6656.  Sums are fp32: within a lane in
// column order, then across lanes in a fixed order, so results repeat bit for bit.
#include <hip/hip_runtime.h>
#include <algorithm>
#include <stdint.h>

#include "ce_device.h"
#include "head_internal.h"

namespace lce {
namespace {

using dev::Elt;
using dev::u32x4;

constexpr float kE4m3Max = 448.0f;
// The smallest scale: its reciprocal is finite.
constexpr float kScaleMin = 1.1754944e-38f;

// 16, 8 and 4 bytes at any address
typedef uint32_t any16 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t any8 __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t any4 __attribute__((aligned(1)));

// E values of a row as loaded, from element index i; the `left` values before the row's end, zeros after
template <bool BF16>
__device__ __forceinline__ u32x4 load_raw(const void *p, int64_t i, int left) {
    constexpr int E = Elt<BF16>::E;
    const char *at = static_cast<const char *>(p) + i * Elt<BF16>::bytes;
    if (left >= E) return *reinterpret_cast<const any16 *>(at);
    float v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = e < left ? Elt<BF16>::load_one(at, e) : 0.0f;
    return Elt<BF16>::pack(v);
}
// LATER: nobody reads them soon, so they need not stay in the caches
template <bool BF16, bool LATER = false>
__device__ __forceinline__ void store_vals(void *p, int64_t i, int left, const float (&v)[Elt<BF16>::E]) {
    constexpr int E = Elt<BF16>::E;
    char *at = static_cast<char *>(p) + i * Elt<BF16>::bytes;
    if (left >= E) {
        const any16 q = Elt<BF16>::pack(v);
        if constexpr (LATER) __builtin_nontemporal_store(q, reinterpret_cast<any16 *>(at));
        else *reinterpret_cast<any16 *>(at) = q;
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (e < left) Elt<BF16>::store_one(at, e, v[e]);
    }
}
// the value as the stream's type holds it
template <bool BF16>
__device__ __forceinline__ float rounded(float v) {
    if constexpr (BF16) return static_cast<float>(static_cast<__bf16>(v));
    else return v;
}
// E weights from column c, plus the offset; ones without a weight
template <int E>
__device__ __forceinline__ void load_weight(const void *w, bool w_bf16, float offset, int c, int left, float (&v)[E]) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = 1.0f;
        return;
    }
    if (left < E) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            v[e] = e >= left ? 0.0f : (w_bf16 ? Elt<true>::load_one(w, c + e) : static_cast<const float *>(w)[c + e]);
    } else if (w_bf16) {
        const char *at = static_cast<const char *>(w) + c * 2;
        if constexpr (E == 8) {
            const u32x4 q = *reinterpret_cast<const any16 *>(at);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = Elt<true>::get(q, e);
        } else {
            const any8 q = *reinterpret_cast<const any8 *>(at);
            v[0] = __uint_as_float(q.x << 16);
            v[1] = __uint_as_float(q.x & 0xffff0000u);
            v[2] = __uint_as_float(q.y << 16);
            v[3] = __uint_as_float(q.y & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            const u32x4 q = *reinterpret_cast<const any16 *>(static_cast<const float *>(w) + c + e);
#pragma unroll
            for (int u = 0; u < 4; ++u) v[e + u] = Elt<false>::get(q, u);
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] += offset;
}

// Sum or maximum over the LPR lanes of a row; the same value in every lane.  The
// LDS slots of two calls with no barrier between their uses must differ.
template <int LPR>
__device__ __forceinline__ float row_sum(float v, float *sh) {
    if constexpr (LPR == 16) {
        v += dev::dpp_f<dev::kDppXor1>(v);
        v += dev::dpp_f<dev::kDppXor2>(v);
        v += dev::dpp_f<dev::kDppHalfMirror>(v);
        v += dev::dpp_f<dev::kDppMirror>(v);
        return v;
    } else {
        v = dev::wave_sum_dpp(v);
        if constexpr (LPR > 64) {
            if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
            __syncthreads();
            v = sh[0];
#pragma unroll
            for (int w = 1; w < LPR / 64; ++w) v += sh[w];
        }
        return v;
    }
}
template <int LPR>
__device__ __forceinline__ float row_max(float v, float *sh) {
    v = fmaxf(v, dev::dpp_f<dev::kDppXor1>(v));
    v = fmaxf(v, dev::dpp_f<dev::kDppXor2>(v));
    v = fmaxf(v, dev::dpp_f<dev::kDppHalfMirror>(v));
    v = fmaxf(v, dev::dpp_f<dev::kDppMirror>(v));
    if constexpr (LPR > 16) {
        v = fmaxf(fmaxf(dev::lane_f(v, 0), dev::lane_f(v, 16)), fmaxf(dev::lane_f(v, 32), dev::lane_f(v, 48)));
        if constexpr (LPR > 64) {
            if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
            __syncthreads();
            v = sh[0];
#pragma unroll
            for (int w = 1; w < LPR / 64; ++w) v = fmaxf(v, sh[w]);
        }
    }
    return v;
}

constexpr int threads_of(int lpr) { return lpr < 256 ? 256 : lpr; }

template <bool BF16, bool OUT8, int LPR, int K>
__global__ __launch_bounds__(threads_of(LPR)) void rms_norm_kernel(NormArgs a) {
    constexpr int E = Elt<BF16>::E, ROWS = threads_of(LPR) / LPR;
    __shared__ float sh[2][16];
    const int lane = threadIdx.x % LPR;
    const int64_t row = a.row0 + static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / LPR;
    if (row >= a.n) return;   // whole rows leave; with LPR >= 256 a workgroup is one row of the grid
    const int H = static_cast<int>(a.H);
    u32x4 x[K], r[K];
    float s[K][E], w[K][E];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * LPR + lane) * E;
        x[k] = r[k] = (u32x4){0u, 0u, 0u, 0u};
        if (c >= H) continue;
        x[k] = load_raw<BF16>(a.x, row * a.ldx + c, H - c);
        if (a.residual) r[k] = load_raw<BF16>(a.residual, row * a.ldr + c, H - c);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * LPR + lane) * E;
        if (c < H) load_weight<E>(a.weight, a.weight_bf16, a.offset, c, H - c, w[k]);
    }
    float q = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * LPR + lane) * E;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            s[k][e] = Elt<BF16>::get(x[k], e);
            if (a.residual) s[k][e] = rounded<BF16>(s[k][e] + Elt<BF16>::get(r[k], e));
        }
        // The sum's next reader comes after the layer that reads y, or in the backward: its stores stream past
        // the caches (8192 x 6656 to 8 bits 71 -> 64 us, 1024 x 4096 7.2 -> 6.3 us; a norm, two products and
        // the addition of the sum after them take the same time either way).  y streamed costs its reader
        // what the norm gains: 8 bits 64 -> 60 us, the product that reads them 10 us more.
        if (a.sum && c < H) store_vals<BF16, true>(a.sum, row * a.lds + c, H - c, s[k]);
#pragma unroll
        for (int e = 0; e < E; ++e) q = fmaf(s[k][e], s[k][e], q);
    }
    q = row_sum<LPR>(q, sh[0]);
    // one square root and one division per row: correctly rounded ones
    const float rstd = 1.0f / sqrtf(q / static_cast<float>(H) + a.eps);
    if (a.rstd && lane == 0) a.rstd[row] = rstd;
    if constexpr (!OUT8) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * LPR + lane) * E;
            if (c >= H) continue;
#pragma unroll
            for (int e = 0; e < E; ++e) s[k][e] = s[k][e] * rstd * w[k][e];
            store_vals<BF16>(a.y, row * a.ldy + c, H - c, s[k]);
        }
    } else {
        float m = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * LPR + lane) * E;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (c < H) s[k][e] = c + e < H ? s[k][e] * rstd * w[k][e] : 0.0f;
                m = fmaxf(m, fabsf(s[k][e]));
            }
        }
        m = row_max<LPR>(m, sh[1]);
        const float scale = m > 0.0f ? fmaxf(m / kE4m3Max, kScaleMin) : 1.0f;
        const float inv = 1.0f / scale;
        if (lane == 0) a.scale[row] = scale;
        unsigned char *y = static_cast<unsigned char *>(a.y) + row * a.ldy;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * LPR + lane) * E;
            if (c >= H) continue;
            uint32_t o[E / 4];
#pragma unroll
            for (int u = 0; u < E / 4; ++u) {
                int p = __builtin_amdgcn_cvt_pk_fp8_f32(s[k][4 * u] * inv, s[k][4 * u + 1] * inv, 0, false);
                p = __builtin_amdgcn_cvt_pk_fp8_f32(s[k][4 * u + 2] * inv, s[k][4 * u + 3] * inv, p, true);
                o[u] = static_cast<uint32_t>(p);
            }
            if (H - c < E) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (c + e < H) y[c + e] = static_cast<unsigned char>(o[e / 4] >> (e % 4 * 8));
            } else if constexpr (E == 8) {
                *reinterpret_cast<any8 *>(y + c) = (any8){o[0], o[1]};
            } else {
                *reinterpret_cast<any4 *>(y + c) = o[0];
            }
        }
    }
}

// A workgroup walks rows blockIdx, blockIdx + gridDim, ... (groups of ROWS) and
// keeps its part of dL/dw in registers, one fp32 sum per column.  The next row's
// values are requested before this row is reduced and stored.  They wait as
// loaded, not widened, so that sixteen waves fit a CU: 8192 x 6656 bf16 takes
// 136 us with widened rows, no request ahead and twelve waves.  With TAIL and two
// accesses a lane the value-by-value branches of every operand take more registers
// than that leaves: bf16 129 of them with a wave a row (twelve waves a CU) and 182
// with 512 lanes (eight); with 1024 lanes 44 are spilled, and 50 of fp32's four accesses.
template <bool BF16, int LPR, int K, bool TAIL>   // TAIL: the last access of a row reaches past its end
__global__ __launch_bounds__(threads_of(LPR)) void rms_norm_backward_kernel(NormGradArgs a) {
    constexpr int E = Elt<BF16>::E, ROWS = threads_of(LPR) / LPR;
    // more accesses per lane leave no registers for another row
    constexpr bool AHEAD = K <= (TAIL ? 1 : 2);
    struct Row {
        u32x4 s[K], g[K], d[K];
        float rstd;
    };
    __shared__ float sh[2][16];
    __shared__ float fold[ROWS > 1 ? ROWS * LPR * K * E : 1];
    const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
    const int H = static_cast<int>(a.H);
    const float inv_h = 1.0f / static_cast<float>(H);
    auto left = [&](int c) { return TAIL ? H - c : E; };   // values of the access before the row's end
    auto fetch = [&](int64_t row, Row &v) {   // zeros past the last row and past H
        v.rstd = row < a.n ? a.rstd[row] : 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * LPR + lane) * E;
            v.s[k] = v.g[k] = v.d[k] = (u32x4){0u, 0u, 0u, 0u};
            if (c < H && row < a.n) {
                v.s[k] = load_raw<BF16>(a.s, row * a.lds + c, left(c));
                v.g[k] = load_raw<BF16>(a.gy, row * a.ldg + c, left(c));
                if (AHEAD && a.gs) v.d[k] = load_raw<BF16>(a.gs, row * a.ldgs + c, left(c));
            }
        }
    };
    float gw[K][E];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) gw[k][e] = 0.0f;
    int turn = 0;
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
    Row cur, next;
    if constexpr (AHEAD) fetch(static_cast<int64_t>(blockIdx.x) * ROWS + sub, cur);
    for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * ROWS; row0 < a.n; row0 += step, turn ^= 1) {
        const int64_t row = row0 + sub;
        fetch(AHEAD ? row + step : row, AHEAD ? next : cur);
        const float rstd = cur.rstd;
        float dot = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * LPR + lane) * E;
            if (c >= H) continue;
            float w[E];
            load_weight<E>(a.weight, a.weight_bf16, a.offset, c, left(c), w);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float sv = Elt<BF16>::get(cur.s[k], e), gv = Elt<BF16>::get(cur.g[k], e);
                gw[k][e] = fmaf(gv, sv * rstd, gw[k][e]);
                dot = fmaf(gv * w[e], sv, dot);
            }
        }
        dot = row_sum<LPR>(dot, sh[turn]);
        const float t = rstd * rstd * (dot * inv_h);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * LPR + lane) * E;
            if (c >= H || row >= a.n) continue;
            float w[E], o[E];
            load_weight<E>(a.weight, a.weight_bf16, a.offset, c, left(c), w);
            if (!AHEAD && a.gs) cur.d[k] = load_raw<BF16>(a.gs, row * a.ldgs + c, left(c));
#pragma unroll
            for (int e = 0; e < E; ++e)
                o[e] = fmaf(rstd, fmaf(-Elt<BF16>::get(cur.s[k], e), t, Elt<BF16>::get(cur.g[k], e) * w[e]),
                            Elt<BF16>::get(cur.d[k], e));
            store_vals<BF16>(a.gx, row * a.ldgx + c, left(c), o);
        }
        if constexpr (AHEAD) cur = next;
    }
    if (!a.gw) return;
    float *part = a.part + static_cast<int64_t>(blockIdx.x) * H;
    if constexpr (ROWS == 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * LPR + lane) * E;
            if (c >= H) continue;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (!TAIL || c + e < H) part[c + e] = gw[k][e];
        }
    } else {
        constexpr int W = LPR * K * E;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < E; ++e) fold[sub * W + (k * LPR + lane) * E + e] = gw[k][e];
        __syncthreads();
        for (int c = threadIdx.x; c < H; c += threads_of(LPR)) {
            float v = fold[c];
#pragma unroll
            for (int r = 1; r < ROWS; ++r) v += fold[r * W + c];
            part[c] = v;
        }
    }
}

// 32 columns per workgroup, eight row groups of 32 threads each
__global__ __launch_bounds__(256) void column_fold_kernel(const float *part, int64_t rows, int64_t ld, int64_t cols,
                                                          void *out, bool out_bf16) {
    __shared__ float sh[8][32];
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x & 31);
    const int r = threadIdx.x >> 5;
    float v = 0.0f;
    if (c < cols) {
        int64_t i = r;
        for (; i + 24 < rows; i += 32) {
            const float p0 = part[i * ld + c], p1 = part[(i + 8) * ld + c], p2 = part[(i + 16) * ld + c],
                        p3 = part[(i + 24) * ld + c];
            v += (p0 + p1) + (p2 + p3);
        }
        for (; i < rows; i += 8) v += part[i * ld + c];
    }
    sh[r][threadIdx.x & 31] = v;
    __syncthreads();
    if (r == 0 && c < cols) {
#pragma unroll
        for (int k = 1; k < 8; ++k) v += sh[k][threadIdx.x];
        if (out_bf16) Elt<true>::store_one(out, c, v);
        else static_cast<float *>(out)[c] = v;
    }
}

// The shape of a row: lanes and accesses per lane.
struct Plan {
    int lpr, k;
};
// Lanes by the number of accesses a row has: a 16-lane group for head-sized rows (four rows per wave),
// then as many lanes as keep one or two accesses each: a row's time is one load, one reduction and one
// store, and short ones keep more rows in flight.  Forward, residual, bf16, the sum stored as y is:
// 16384 x 1536 35 us with 256 lanes of one access, 41 with a wave of four; 16384 x 4096 91 us with 512 of
// one, 99 with 256 of two; 8192 x 6656 83 us with 512 of two, 93 with 256 of four; 16384 x 1024 22 us with
// a wave of two, 24 with 256 of one.
Plan plan_of(int64_t H, int e) {
    const int64_t nv = (H + e - 1) / e;
    if (nv <= 16) return {16, 1};
    if (nv <= 64) return {64, 1};
    if (nv <= 128) return {64, 2};
    if (nv <= 256) return {256, 1};
    if (nv <= 512) return {512, 1};
    if (nv <= 1024) return {512, 2};
    if (nv <= 2048) return {1024, 2};
    return {1024, 4};
}

template <bool BF16, bool OUT8, int LPR, int K>
void launch_fwd(const NormArgs &a, hipStream_t st) {
    constexpr int ROWS = threads_of(LPR) / LPR;
    // a launch has fewer than 2^32 threads: at most 2^21 workgroups at a time
    constexpr int64_t kRows = (int64_t(1) << 21) * ROWS;
    for (NormArgs b = a; b.row0 < a.n; b.row0 += kRows) {
        const unsigned grid = static_cast<unsigned>((std::min(a.n - b.row0, kRows) + ROWS - 1) / ROWS);
        hipLaunchKernelGGL((rms_norm_kernel<BF16, OUT8, LPR, K>), dim3(grid), dim3(threads_of(LPR)), 0, st, b);
    }
}
template <bool BF16, bool OUT8>
void pick_fwd(const NormArgs &a, hipStream_t st) {
    const Plan p = plan_of(a.H, Elt<BF16>::E);
    if (p.lpr == 16) launch_fwd<BF16, OUT8, 16, 1>(a, st);
    else if (p.lpr == 64 && p.k == 1) launch_fwd<BF16, OUT8, 64, 1>(a, st);
    else if (p.lpr == 64) launch_fwd<BF16, OUT8, 64, 2>(a, st);
    else if (p.lpr == 256) launch_fwd<BF16, OUT8, 256, 1>(a, st);
    else if (p.lpr == 512 && p.k == 1) launch_fwd<BF16, OUT8, 512, 1>(a, st);
    else if (p.lpr == 512) launch_fwd<BF16, OUT8, 512, 2>(a, st);
    else if (BF16 || p.k == 2) launch_fwd<BF16, OUT8, 1024, 2>(a, st);
    else launch_fwd<BF16, OUT8, 1024, BF16 ? 2 : 4>(a, st);   // fp32 only: bf16 rows end at 2048 accesses
}

template <bool BF16, int LPR, int K>
int64_t launch_bwd(const NormGradArgs &a, hipStream_t st) {
    constexpr int ROWS = threads_of(LPR) / LPR;
    // Sixteen waves on every compute unit, and few partial rows.  Without TAIL all groups run at once; where
    // a kernel's registers leave fewer waves the rest of the groups follow.
    const int64_t most = std::min<int64_t>(kNormMaxGroups, static_cast<int64_t>(device_cu_count()) * (1024 / threads_of(LPR)));
    const int64_t groups = std::min((a.n + ROWS - 1) / ROWS, most);
    const dim3 grid(static_cast<unsigned>(groups)), block(threads_of(LPR));
    if (a.H % Elt<BF16>::E) hipLaunchKernelGGL((rms_norm_backward_kernel<BF16, LPR, K, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((rms_norm_backward_kernel<BF16, LPR, K, false>), grid, block, 0, st, a);
    return groups;
}
template <bool BF16>
int64_t pick_bwd(const NormGradArgs &a, hipStream_t st) {
    const Plan p = plan_of(a.H, Elt<BF16>::E);
    if (p.lpr == 16) return launch_bwd<BF16, 16, 1>(a, st);
    if (p.lpr == 64 && p.k == 1) return launch_bwd<BF16, 64, 1>(a, st);
    if (p.lpr == 64) return launch_bwd<BF16, 64, 2>(a, st);
    if (p.lpr == 256) return launch_bwd<BF16, 256, 1>(a, st);
    if (p.lpr == 512 && p.k == 1) return launch_bwd<BF16, 512, 1>(a, st);
    if (p.lpr == 512) return launch_bwd<BF16, 512, 2>(a, st);
    if (BF16 || p.k == 2) return launch_bwd<BF16, 1024, 2>(a, st);
    return launch_bwd<BF16, 1024, BF16 ? 2 : 4>(a, st);   // fp32 only
}

}  // namespace

hipError_t launch_column_fold(const float *part, int64_t rows, int64_t ld, int64_t cols, void *out, bool out_bf16,
                              hipStream_t st) {
    if (cols <= 0) return hipSuccess;
    hipLaunchKernelGGL(column_fold_kernel, dim3(static_cast<unsigned>((cols + 31) / 32)), dim3(256), 0, st, part, rows,
                       ld, cols, out, out_bf16);
    return hipGetLastError();
}

hipError_t launch_rms_norm(const NormArgs &a, bool is_bf16, hipStream_t st) {
    if (a.n == 0) return hipSuccess;
    if (is_bf16) a.out8 ? pick_fwd<true, true>(a, st) : pick_fwd<true, false>(a, st);
    else a.out8 ? pick_fwd<false, true>(a, st) : pick_fwd<false, false>(a, st);
    return hipGetLastError();
}

hipError_t launch_rms_norm_backward(const NormGradArgs &a, bool is_bf16, hipStream_t st) {
    int64_t groups = 0;
    if (a.n > 0) {
        groups = is_bf16 ? pick_bwd<true>(a, st) : pick_bwd<false>(a, st);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!a.gw) return hipSuccess;
    return launch_column_fold(a.part, groups, a.H, a.H, a.gw, a.gw_bf16, st);   // n = 0: zeros
}

}  // namespace lce
