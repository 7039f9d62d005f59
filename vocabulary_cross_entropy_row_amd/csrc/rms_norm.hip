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
// lives in the registers of LPR lanes (16, 64, 256 or 1024) between its load and
// its stores, K accesses of E values per lane: 16 bytes where the rows and their
// strides allow it, single values otherwise.  Sums are fp32: within a lane in
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

// E values of a row in the type, from element index i (16-byte aligned when E > 1)
template <bool BF16, int E>
__device__ __forceinline__ void load_vals(const void *p, int64_t i, float (&v)[E]) {
    if constexpr (E == 1) {
        v[0] = Elt<BF16>::load_one(p, i);
    } else {
        const u32x4 q = *reinterpret_cast<const u32x4 *>(static_cast<const char *>(p) + i * Elt<BF16>::bytes);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = Elt<BF16>::get(q, e);
    }
}
template <bool BF16, int E>
__device__ __forceinline__ void store_vals(void *p, int64_t i, const float (&v)[E]) {
    if constexpr (E == 1) Elt<BF16>::store_one(p, i, v[0]);
    else *reinterpret_cast<u32x4 *>(static_cast<char *>(p) + i * Elt<BF16>::bytes) = Elt<BF16>::pack(v);
}
// the value as the stream's type holds it
template <bool BF16>
__device__ __forceinline__ float rounded(float v) {
    if constexpr (BF16) return static_cast<float>(static_cast<__bf16>(v));
    else return v;
}
// E weights from column c, plus the offset; ones without a weight
template <int E>
__device__ __forceinline__ void load_weight(const void *w, bool w_bf16, float offset, int c, float (&v)[E]) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = 1.0f;
        return;
    }
    if (w_bf16) {
        if constexpr (E == 8) {
            load_vals<true, 8>(w, c, v);
        } else if constexpr (E == 4) {
            const uint2 q = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(w) + c);
            v[0] = __uint_as_float(q.x << 16);
            v[1] = __uint_as_float(q.x & 0xffff0000u);
            v[2] = __uint_as_float(q.y << 16);
            v[3] = __uint_as_float(q.y & 0xffff0000u);
        } else {
            v[0] = Elt<true>::load_one(w, c);
        }
    } else {
        const float *f = static_cast<const float *>(w) + c;
        if constexpr (E == 1) {
            v[0] = f[0];
        } else {
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                const float4 q = *reinterpret_cast<const float4 *>(f + e);
                v[e] = q.x;
                v[e + 1] = q.y;
                v[e + 2] = q.z;
                v[e + 3] = q.w;
            }
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

template <bool BF16, bool OUT8, int E, int LPR, int K>
__global__ __launch_bounds__(threads_of(LPR)) void rms_norm_kernel(NormArgs a) {
    constexpr int ROWS = threads_of(LPR) / LPR;
    __shared__ float sh[2][16];
    const int lane = threadIdx.x % LPR;
    const int64_t row = a.row0 + static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / LPR;
    if (row >= a.n) return;   // whole rows leave; with LPR >= 256 a workgroup is one row of the grid
    const int H = static_cast<int>(a.H);
    float s[K][E], w[K][E];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * LPR + lane) * E;
#pragma unroll
        for (int e = 0; e < E; ++e) s[k][e] = 0.0f;
        if (c < H) load_vals<BF16, E>(a.x, row * a.ldx + c, s[k]);
    }
    if (a.residual) {
        float r[K][E];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * LPR + lane) * E;
#pragma unroll
            for (int e = 0; e < E; ++e) r[k][e] = 0.0f;
            if (c < H) load_vals<BF16, E>(a.residual, row * a.ldr + c, r[k]);
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < E; ++e) s[k][e] = rounded<BF16>(s[k][e] + r[k][e]);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * LPR + lane) * E;
        if (c < H) load_weight<E>(a.weight, a.weight_bf16, a.offset, c, w[k]);
    }
    float q = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * LPR + lane) * E;
        if (a.sum && c < H) store_vals<BF16, E>(a.sum, row * a.lds + c, s[k]);
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
            store_vals<BF16, E>(a.y, row * a.ldy + c, s[k]);
        }
    } else {
        float m = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * LPR + lane) * E;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (c < H) s[k][e] = s[k][e] * rstd * w[k][e];
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
            if constexpr (E == 1) {
                y[c] = static_cast<unsigned char>(__builtin_amdgcn_cvt_pk_fp8_f32(s[k][0] * inv, 0.0f, 0, false));
            } else {
                uint32_t o[E / 4];
#pragma unroll
                for (int u = 0; u < E / 4; ++u) {
                    int p = __builtin_amdgcn_cvt_pk_fp8_f32(s[k][4 * u] * inv, s[k][4 * u + 1] * inv, 0, false);
                    p = __builtin_amdgcn_cvt_pk_fp8_f32(s[k][4 * u + 2] * inv, s[k][4 * u + 3] * inv, p, true);
                    o[u] = static_cast<uint32_t>(p);
                }
                if constexpr (E == 8) *reinterpret_cast<uint2 *>(y + c) = make_uint2(o[0], o[1]);
                else *reinterpret_cast<uint32_t *>(y + c) = o[0];
            }
        }
    }
}

// An access of a row as loaded: 16 bytes, or one widened value
template <int E>
struct Raw { typedef u32x4 type; };
template <>
struct Raw<1> { typedef float type; };
template <bool BF16, int E>
__device__ __forceinline__ typename Raw<E>::type load_raw(const void *p, int64_t i) {
    if constexpr (E == 1) return Elt<BF16>::load_one(p, i);
    else return *reinterpret_cast<const u32x4 *>(static_cast<const char *>(p) + i * Elt<BF16>::bytes);
}
template <bool BF16, int E>
__device__ __forceinline__ float raw_get(const typename Raw<E>::type &v, int e) {
    if constexpr (E == 1) return v;
    else return Elt<BF16>::get(v, e);
}

// A workgroup walks rows blockIdx, blockIdx + gridDim, ... (groups of ROWS) and
// keeps its part of dL/dw in registers, one fp32 sum per column.  The next row's
// values are requested before this row is reduced and stored.  They wait as
// loaded, not widened, so that sixteen waves fit a CU: 8192 x 6656 bf16 takes
// 136 us with widened rows, no request ahead and twelve waves.
template <bool BF16, int E, int LPR, int K>
__global__ __launch_bounds__(threads_of(LPR)) void rms_norm_backward_kernel(NormGradArgs a) {
    constexpr int ROWS = threads_of(LPR) / LPR;
    typedef typename Raw<E>::type raw;
    // shapes with more accesses per lane have no registers left for another row
    constexpr bool AHEAD = E > 1 ? K <= 2 : K <= 4;
    struct Row {
        raw s[K], g[K], d[K];
        float rstd;
    };
    __shared__ float sh[2][16];
    __shared__ float fold[ROWS > 1 ? ROWS * LPR * K * E : 1];
    const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
    const int H = static_cast<int>(a.H);
    const float inv_h = 1.0f / static_cast<float>(H);
    auto fetch = [&](int64_t row, Row &v) {   // zeros past the last row and past H
        v.rstd = row < a.n ? a.rstd[row] : 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * LPR + lane) * E;
            v.s[k] = v.g[k] = v.d[k] = raw{};
            if (c < H && row < a.n) {
                v.s[k] = load_raw<BF16, E>(a.s, row * a.lds + c);
                v.g[k] = load_raw<BF16, E>(a.gy, row * a.ldg + c);
                if (AHEAD && a.gs) v.d[k] = load_raw<BF16, E>(a.gs, row * a.ldgs + c);
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
            load_weight<E>(a.weight, a.weight_bf16, a.offset, c, w);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float sv = raw_get<BF16, E>(cur.s[k], e), gv = raw_get<BF16, E>(cur.g[k], e);
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
            load_weight<E>(a.weight, a.weight_bf16, a.offset, c, w);
            if (!AHEAD && a.gs) cur.d[k] = load_raw<BF16, E>(a.gs, row * a.ldgs + c);
#pragma unroll
            for (int e = 0; e < E; ++e)
                o[e] = fmaf(rstd, fmaf(-raw_get<BF16, E>(cur.s[k], e), t, raw_get<BF16, E>(cur.g[k], e) * w[e]),
                            raw_get<BF16, E>(cur.d[k], e));
            store_vals<BF16, E>(a.gx, row * a.ldgx + c, o);
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
            for (int e = 0; e < E; ++e) part[c + e] = gw[k][e];
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

// The shape of a row: values per access, lanes and accesses per lane.
struct Plan {
    int e, lpr, k;
};
// Lanes by the number of accesses a row has: a 16-lane group for head-sized rows (four rows per wave),
// then as many lanes as keep one or two accesses each: a row's time is one load, one reduction and one
// store, and short ones keep more rows in flight.  Forward, residual, bf16: 16384 x 1536 35 us with 256
// lanes of one access, 41 with a wave of four; 16384 x 4096 91 us with 512 of one, 99 with 256 of two;
// 8192 x 6656 83 us with 512 of two, 93 with 256 of four; 16384 x 1024 22 us with a wave of two, 24
// with 256 of one.
Plan plan_of(int64_t H, bool vec, int e) {
    if (!vec) {
        if (H <= 256) return {1, 64, 4};
        if (H <= 2048) return {1, 256, 8};
        if (H <= 8192) return {1, 1024, 8};
        return {1, 1024, 16};
    }
    const int64_t nv = H / e;
    if (nv <= 16) return {e, 16, 1};
    if (nv <= 64) return {e, 64, 1};
    if (nv <= 128) return {e, 64, 2};
    if (nv <= 256) return {e, 256, 1};
    if (nv <= 512) return {e, 512, 1};
    if (nv <= 1024) return {e, 512, 2};
    if (nv <= 2048) return {e, 1024, 2};
    return {e, 1024, 4};
}

bool on16(const void *p, int64_t ld, int bytes) {
    return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * bytes) % 16 == 0);
}

template <bool BF16, bool OUT8, int E, int LPR, int K>
void launch_fwd(const NormArgs &a, hipStream_t st) {
    constexpr int ROWS = threads_of(LPR) / LPR;
    // a launch has fewer than 2^32 threads: at most 2^21 workgroups at a time
    constexpr int64_t kRows = (int64_t(1) << 21) * ROWS;
    for (NormArgs b = a; b.row0 < a.n; b.row0 += kRows) {
        const unsigned grid = static_cast<unsigned>((std::min(a.n - b.row0, kRows) + ROWS - 1) / ROWS);
        hipLaunchKernelGGL((rms_norm_kernel<BF16, OUT8, E, LPR, K>), dim3(grid), dim3(threads_of(LPR)), 0, st, b);
    }
}
template <bool BF16, bool OUT8, int E>
void pick_fwd(const NormArgs &a, const Plan &p, hipStream_t st) {
    if constexpr (E == 1) {
        if (p.lpr == 64) launch_fwd<BF16, OUT8, 1, 64, 4>(a, st);
        else if (p.lpr == 256) launch_fwd<BF16, OUT8, 1, 256, 8>(a, st);
        else if (p.k == 8) launch_fwd<BF16, OUT8, 1, 1024, 8>(a, st);
        else launch_fwd<BF16, OUT8, 1, 1024, 16>(a, st);
    } else {
        if (p.lpr == 16) launch_fwd<BF16, OUT8, E, 16, 1>(a, st);
        else if (p.lpr == 64 && p.k == 1) launch_fwd<BF16, OUT8, E, 64, 1>(a, st);
        else if (p.lpr == 64) launch_fwd<BF16, OUT8, E, 64, 2>(a, st);
        else if (p.lpr == 256) launch_fwd<BF16, OUT8, E, 256, 1>(a, st);
        else if (p.lpr == 512 && p.k == 1) launch_fwd<BF16, OUT8, E, 512, 1>(a, st);
        else if (p.lpr == 512) launch_fwd<BF16, OUT8, E, 512, 2>(a, st);
        else if (E == 8 || p.k == 2) launch_fwd<BF16, OUT8, E, 1024, 2>(a, st);
        else launch_fwd<BF16, OUT8, E, 1024, E == 8 ? 2 : 4>(a, st);   // fp32 only: bf16 rows end at 2048 accesses
    }
}

template <bool BF16, int E, int LPR, int K>
void launch_bwd(const NormGradArgs &a, hipStream_t st, int64_t *groups) {
    constexpr int ROWS = threads_of(LPR) / LPR;
    const int64_t want = (a.n + ROWS - 1) / ROWS;
    // sixteen waves on every compute unit: all groups run at once, and few partial rows
    const int64_t most = std::min<int64_t>(kNormMaxGroups, static_cast<int64_t>(device_cu_count()) * (1024 / threads_of(LPR)));
    *groups = std::min(want, most);
    hipLaunchKernelGGL((rms_norm_backward_kernel<BF16, E, LPR, K>), dim3(static_cast<unsigned>(*groups)),
                       dim3(threads_of(LPR)), 0, st, a);
}
template <bool BF16, int E>
void pick_bwd(const NormGradArgs &a, const Plan &p, hipStream_t st, int64_t *groups) {
    if constexpr (E == 1) {
        if (p.lpr == 64) launch_bwd<BF16, 1, 64, 4>(a, st, groups);
        else if (p.lpr == 256) launch_bwd<BF16, 1, 256, 8>(a, st, groups);
        else if (p.k == 8) launch_bwd<BF16, 1, 1024, 8>(a, st, groups);
        else launch_bwd<BF16, 1, 1024, 16>(a, st, groups);
    } else {
        if (p.lpr == 16) launch_bwd<BF16, E, 16, 1>(a, st, groups);
        else if (p.lpr == 64 && p.k == 1) launch_bwd<BF16, E, 64, 1>(a, st, groups);
        else if (p.lpr == 64) launch_bwd<BF16, E, 64, 2>(a, st, groups);
        else if (p.lpr == 256) launch_bwd<BF16, E, 256, 1>(a, st, groups);
        else if (p.lpr == 512 && p.k == 1) launch_bwd<BF16, E, 512, 1>(a, st, groups);
        else if (p.lpr == 512) launch_bwd<BF16, E, 512, 2>(a, st, groups);
        else if (E == 8 || p.k == 2) launch_bwd<BF16, E, 1024, 2>(a, st, groups);
        else launch_bwd<BF16, E, 1024, E == 8 ? 2 : 4>(a, st, groups);   // fp32 only
    }
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
    const int es = is_bf16 ? 2 : 4, e = 16 / es;
    const bool vec = a.H % e == 0 && on16(a.x, a.ldx, es) && on16(a.residual, a.ldr, es) && on16(a.sum, a.lds, es) &&
                     on16(a.weight, 0, 1) && (a.out8 ? reinterpret_cast<uintptr_t>(a.y) % 8 == 0 && a.ldy % 8 == 0
                                                     : on16(a.y, a.ldy, es));
    const Plan p = plan_of(a.H, vec, e);
    if (is_bf16) {
        if (a.out8) vec ? pick_fwd<true, true, 8>(a, p, st) : pick_fwd<true, true, 1>(a, p, st);
        else vec ? pick_fwd<true, false, 8>(a, p, st) : pick_fwd<true, false, 1>(a, p, st);
    } else {
        if (a.out8) vec ? pick_fwd<false, true, 4>(a, p, st) : pick_fwd<false, true, 1>(a, p, st);
        else vec ? pick_fwd<false, false, 4>(a, p, st) : pick_fwd<false, false, 1>(a, p, st);
    }
    return hipGetLastError();
}

hipError_t launch_rms_norm_backward(const NormGradArgs &a, bool is_bf16, hipStream_t st) {
    int64_t groups = 0;
    if (a.n > 0) {
        const int es = is_bf16 ? 2 : 4, e = 16 / es;
        const bool vec = a.H % e == 0 && on16(a.gy, a.ldg, es) && on16(a.s, a.lds, es) && on16(a.gs, a.ldgs, es) &&
                         on16(a.gx, a.ldgx, es) && on16(a.weight, 0, 1);
        const Plan p = plan_of(a.H, vec, e);
        if (is_bf16) vec ? pick_bwd<true, 8>(a, p, st, &groups) : pick_bwd<true, 1>(a, p, st, &groups);
        else vec ? pick_bwd<false, 4>(a, p, st, &groups) : pick_bwd<false, 1>(a, p, st, &groups);
        const hipError_t e2 = hipGetLastError();
        if (e2 != hipSuccess) return e2;
    }
    if (!a.gw) return hipSuccess;
    return launch_column_fold(a.part, groups, a.H, a.H, a.gw, a.gw_bf16, st);   // n = 0: zeros
}

}  // namespace lce
