// Matrix product with an epilogue on the gfx950 matrix cores:
//   z[t, f] = scale_x[t] scale_w[f] sum_k x[t, k] w[f, k] + bias[f]
//   out     = act(z) + residual
// for bf16 or e4m3 operands with K contiguous, fp32 accumulation, output bf16 or
// fp32.
//
// A workgroup computes a tile of BF features (rows of w) by BT tokens.  K advances
// in steps of 128 bytes per row; both operands' tiles of a step go straight from
// memory to LDS (buffer->LDS loads of 1 KB per wave: 8 rows x 128 bytes), SA steps
// of w and SB steps of x in flight or in use.  One barrier per step hands the tiles
// over.  Row r of a tile keeps its 16-byte chunk c at position c ^ (r / 2 mod 8),
// so a fragment read (32 consecutive rows, one chunk) spreads over all banks.
//
// The features are the rows of the MFMA (its A operand) and the tokens its columns,
// so a lane's accumulators are runs of four consecutive features of one token.  The
// epilogue passes each wave's tile through LDS, 32 tokens at a time, and takes eight
// consecutive features per lane: bias and scales are read once per lane, and
// residual, pre-activation and output move 16 bytes at a time.
//
// 256 x 256 tiles, 1024 x 6656 x 202048 bf16: 2.2 ms, 1.25 PFLOP/s with the matrix
// units busy 71% of the time at the 1.4 to 1.7 GHz that their power leaves (all-zero
// operands run 1.4 times as fast); the library product of 8192 to 16384 cubed reaches
// 1.42 to 1.55.  A step of K takes 1.5 us and a tile's start and end 8 to 10, half of
// that stores, which nothing overlaps.  e4m3, 4096 x 8192 x 8192: 245 us, 2.2 PFLOP/s,
// matrix units busy 47 to 54% at 2.0 to 2.1 GHz; the waves wait for operands (a row stride of 8192
// bytes costs 8% of that; five tiles of 64 bytes in flight instead of 2.5 of 128 gain
// nothing).
//
// MFMA operand layout: lane l supplies row l % 32 of A (column of B) and, of a step
// of K, the 16-byte chunk 2 s + l / 32 for bf16 sub-step s (32x32x16); an e4m3
// sub-step (32x32x64) takes the chunks of two bf16 sub-steps.  Which k a byte stands
// for is the same in both operands, so their order within a step does not matter to
// the sum.  (The e4m3 instructions bring the eight products of a lane's half chunk to
// a unit of 2^-13 of the largest and cut the rest off before they add, whatever the
// accumulator: measured on the device.  A bf16 output rounds 2^4 times coarser, and
// only that is offered for them.)  Result register r of lane l is row (r / 4) 8 + (l / 32) 4 + r % 4,
// column l % 32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ce_device.h"
#include "head_internal.h"

namespace lce {
namespace linear {

using dev::Elt;
using dev::u32x4;

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef float f4v __attribute__((ext_vector_type(4)));
// 16 bytes at any address: gfx950 loads and stores them in one instruction, so rows of odd length cost
// no more than aligned ones (one value per store took 35 us where this takes 26, 77 x 1000 x 50257 with
// fp32 outputs)
typedef uint32_t any16 __attribute__((ext_vector_type(4), aligned(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void *lds_ptr;

constexpr uint32_t kOutside = 0xFFFFFFF0u;   // an offset no descriptor covers: reads zeros

struct Epi {
    const float *scale_x, *scale_w;
    const void *bias;
    bool bias_bf16;
    int act;
    const void *residual;
    int64_t ldr;
    void *out;
    int64_t ldo;
    bool out_bf16, streams;   // streams: a bf16 output is stored past the caches
    void *preact;
    int64_t ldp;
    int64_t n, M;
};

struct Args {
    const unsigned char *w, *x;
    int64_t ldw, ldx;     // bytes
    int kbytes;           // of K per row
    int n, M;
    int tiles_f, tiles_t, splits;
    int per_xcd;          // ceil(tiles * splits / 8)
    float *part;          // splits > 1: partials [splits][n][ldpart]
    int64_t ldpart;
    Epi e;
};

// LDS position of chunk c of row r is c ^ swz(r): the 16 rows that one LDS cycle serves for a fragment
// read (consecutive rows, one chunk) land on 16 distinct 16-byte groups of the 256-byte bank window.
__device__ __forceinline__ int swz(int r) { return (r / 2) & 7; }

// A buffer descriptor built from wave-uniform values, so it lives in SGPRs.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const void *p, uint32_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>((static_cast<uint64_t>(hi) << 32) | lo), 0,
                                             __builtin_amdgcn_readfirstlane(bytes), dev::kBufferWord3);
}

// tanh(u) = 1 - 2 / (1 + e^{2u}), from |u| so that nothing overflows
__device__ __forceinline__ float tanh_fast(float u) {
    const float t = dev::exp2_fast(fabsf(u) * (-2.0f * dev::kLog2e));
    return copysignf((1.0f - t) * dev::rcp_fast(1.0f + t), u);
}
__device__ __forceinline__ float sigmoid_fast(float z) { return dev::rcp_fast(1.0f + dev::exp2_fast(-z * dev::kLog2e)); }

constexpr float kSqrt2OverPi = 0.79788456080286536f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kCubic = 0.044715f;

// The normal distribution function of z, with g = e^{-z^2 / 2}: Abramowitz and Stegun's rational
// approximation 7.1.26 of the complementary error function at |z| / sqrt 2 (absolute error below
// 1.5e-7), taken on the side where nothing cancels.  A tenth of the library function's
// instructions, which would cost the epilogue of a 4096-deep product a fifth of its time.
__device__ __forceinline__ float normal_cdf(float z, float g) {
    const float t = dev::rcp_fast(fmaf(fabsf(z), 0.3275911f * 0.70710678118654752f, 1.0f));
    const float p = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f), -0.284496736f), 0.254829592f);
    const float tail = 0.5f * p * g;
    return z < 0.0f ? tail : 1.0f - tail;
}
__device__ __forceinline__ float gauss(float z) { return dev::exp2_fast(z * z * (-0.5f * dev::kLog2e)); }

__device__ __forceinline__ float activate(int act, float z) {
    switch (act) {   // uniform over the launch
        case ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
        case ACT_GELU: return z * normal_cdf(z, gauss(z));
        case ACT_GELU_TANH: return 0.5f * z * (1.0f + tanh_fast(kSqrt2OverPi * fmaf(kCubic * z * z, z, z)));
        case ACT_SILU: return z * sigmoid_fast(z);
        default: return z;
    }
}
// U x W values: the choice once, not per value
template <int ACT, int U, int W>
__device__ __forceinline__ void activate_all(float (&v)[U][W]) {
#pragma unroll
    for (int p = 0; p < U; ++p)
#pragma unroll
        for (int u = 0; u < W; ++u) v[p][u] = activate(ACT, v[p][u]);
}
template <int U, int W>
__device__ __forceinline__ void activate_block(int act, float (&v)[U][W]) {
    switch (act) {
        case ACT_RELU: activate_all<ACT_RELU>(v); break;
        case ACT_GELU: activate_all<ACT_GELU>(v); break;
        case ACT_GELU_TANH: activate_all<ACT_GELU_TANH>(v); break;
        case ACT_SILU: activate_all<ACT_SILU>(v); break;
        default: break;
    }
}
// d act / dz
__device__ __forceinline__ float slope(int act, float z) {
    switch (act) {
        case ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
        case ACT_GELU: {
            const float g = gauss(z);
            return fmaf(z * kInvSqrt2Pi, g, normal_cdf(z, g));
        }
        case ACT_GELU_TANH: {
            const float t = tanh_fast(kSqrt2OverPi * fmaf(kCubic * z * z, z, z));
            const float q = 1.0f - t * t;   // 0 far out, where z^2 may overflow
            const float bend = q > 0.0f ? 0.5f * z * q * kSqrt2OverPi * fmaf(3.0f * kCubic, z * z, 1.0f) : 0.0f;
            return bend + 0.5f * (1.0f + t);
        }
        case ACT_SILU: {
            const float s = sigmoid_fast(z);
            return s * fmaf(z, 1.0f - s, 1.0f);
        }
        default: return 1.0f;
    }
}

// What a lane keeps for its eight features f .. f + 7
struct Cols {
    float sw[8], b[8];
};
__device__ __forceinline__ Cols load_cols(const Epi &e, int64_t f) {
    Cols c;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        const bool in = f + u < e.M;
        c.sw[u] = e.scale_w && in ? e.scale_w[f + u] : 1.0f;
        c.b[u] = !e.bias || !in ? 0.0f
                                : (e.bias_bf16 ? Elt<true>::load_one(e.bias, f + u) : static_cast<const float *>(e.bias)[f + u]);
    }
    return c;
}
// The sums v of tokens t0, t0 + dt, ... (U of them), features f .. f + 7, through the epilogue to
// memory.  The residuals are requested before the sums are read (read()), so U tokens wait for memory
// once.
template <int U, class Read>
__device__ __forceinline__ void finish(const Epi &e, const Cols &c, int64_t t0, int dt, int64_t f, Read read) {
    const bool vec = f + 8 <= e.M;
    u32x4 ra[U], rb[U];   // the residual's 16 bytes (bf16) or 32 (fp32)
    if (e.residual && vec) {
#pragma unroll
        for (int p = 0; p < U; ++p) {
            const int64_t t = t0 + p * dt;
            ra[p] = rb[p] = (u32x4){0u, 0u, 0u, 0u};
            if (t >= e.n) continue;
            const char *r = static_cast<const char *>(e.residual) + (t * e.ldr + f) * (e.out_bf16 ? 2 : 4);
            ra[p] = reinterpret_cast<const any16 *>(r)[0];
            if (!e.out_bf16) rb[p] = reinterpret_cast<const any16 *>(r)[1];
        }
    }
    float v[U][8];
    read(v);
    if (e.scale_w) {
#pragma unroll
        for (int p = 0; p < U; ++p)
#pragma unroll
            for (int u = 0; u < 8; ++u) v[p][u] *= c.sw[u];
    }
    if (e.bias) {
#pragma unroll
        for (int p = 0; p < U; ++p)
#pragma unroll
            for (int u = 0; u < 8; ++u) v[p][u] += c.b[u];
    }
    if (e.preact) {
#pragma unroll
        for (int p = 0; p < U; ++p) {
            const int64_t t = t0 + p * dt, o = t * e.ldp + f;
            if (t >= e.n) continue;
            if (vec) {
                *reinterpret_cast<any16 *>(static_cast<uint16_t *>(e.preact) + o) = Elt<true>::pack(v[p]);
            } else {
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (f + u < e.M) Elt<true>::store_one(e.preact, o + u, v[p][u]);
            }
        }
    }
    if (e.act != ACT_NONE) activate_block(e.act, v);
    if (vec && e.out_bf16) {
#pragma unroll
        for (int p = 0; p < U; ++p) {
            const int64_t t = t0 + p * dt;
            if (t >= e.n) continue;
            if (e.residual) {
#pragma unroll
                for (int u = 0; u < 8; ++u) v[p][u] += Elt<true>::get(ra[p], u);
            }
            any16 *o = reinterpret_cast<any16 *>(static_cast<uint16_t *>(e.out) + t * e.ldo + f);
            const any16 q = Elt<true>::pack(v[p]);
            if (e.streams) {
                asm volatile("");   // before and after: or the two stores become one that does not stream
                __builtin_nontemporal_store(q, o);
                asm volatile("");
            } else {
                *o = q;
            }
        }
    } else if (vec) {
#pragma unroll
        for (int p = 0; p < U; ++p) {
            const int64_t t = t0 + p * dt;
            if (t >= e.n) continue;
            if (e.residual) {
#pragma unroll
                for (int u = 0; u < 8; ++u) v[p][u] += Elt<false>::get(u < 4 ? ra[p] : rb[p], u & 3);
            }
            any16 *q = reinterpret_cast<any16 *>(static_cast<float *>(e.out) + t * e.ldo + f);
            q[0] = __builtin_bit_cast(u32x4, make_float4(v[p][0], v[p][1], v[p][2], v[p][3]));
            q[1] = __builtin_bit_cast(u32x4, make_float4(v[p][4], v[p][5], v[p][6], v[p][7]));
        }
    } else {
#pragma unroll
        for (int p = 0; p < U; ++p) {
            const int64_t t = t0 + p * dt, o = t * e.ldo + f;
            if (t >= e.n) continue;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (f + u >= e.M) continue;
                if (e.out_bf16) {
                    if (e.residual) v[p][u] += Elt<true>::load_one(e.residual, t * e.ldr + f + u);
                    Elt<true>::store_one(e.out, o + u, v[p][u]);
                } else {
                    if (e.residual) v[p][u] += static_cast<const float *>(e.residual)[t * e.ldr + f + u];
                    static_cast<float *>(e.out)[o + u] = v[p][u];
                }
            }
        }
    }
}

constexpr int kStep = 128;                    // bytes of K per row and step
constexpr int kChunks = kStep / 16;           // 16-byte chunks in them
constexpr int kLoadRows = 1024 / kStep;       // rows that a wave's load of 1 KB takes

// One tile shape: BF x BT by WF x WT waves, SA steps of w and SB of x in LDS.
template <int BF_, int BT_, int WF_, int WT_, int SA_, int SB_>
struct Shape {
    static constexpr int BF = BF_, BT = BT_, WF = WF_, WT = WT_, SA = SA_, SB = SB_;
    static constexpr int NW = WF * WT;
    static constexpr int FI = BF / WF / 32, TJ = BT / WT / 32;      // 32 x 32 tiles per wave
    static constexpr int LA = BF / kLoadRows / NW, LB = BT / kLoadRows / NW;   // 1 KB loads per wave and step
    static constexpr int A_BYTES = BF * kStep, B_BYTES = BT * kStep;
    static constexpr int OUT_LD = FI * 32 + 4;                      // floats per token of a wave's epilogue tile
    static constexpr int LOOP_LDS = SA * A_BYTES + SB * B_BYTES;
    static constexpr int OUT_LDS = NW * 32 * OUT_LD * 4;
    static constexpr int LDS = LOOP_LDS > OUT_LDS ? LOOP_LDS : OUT_LDS;
    static constexpr int PER_CU = 160 * 1024 / LDS < 8 / NW ? 160 * 1024 / LDS : (8 / NW > 0 ? 8 / NW : 1);
    static_assert(FI >= 1 && TJ >= 1 && LA * kLoadRows * NW == BF && LB * kLoadRows * NW == BT && LDS <= 160 * 1024, "tile shape");
    static_assert((SA == SB || SA == SB + 1) && SB >= 2, "steps in flight");
};

template <bool FP8>
struct Frag;
template <>
struct Frag<false> {
    typedef bf8 type;
    static constexpr int BYTES = 32;   // of K per MFMA
    __device__ static __forceinline__ bf8 load(const unsigned char *row, int sw, int kk, int half) {
        return *reinterpret_cast<const bf8 *>(row + ((kk * 2 + half) ^ sw) * 16);
    }
    __device__ static __forceinline__ f16v mfma(bf8 a, bf8 b, f16v c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Frag<true> {
    typedef i32x8 type;
    static constexpr int BYTES = 64;
    __device__ static __forceinline__ i32x8 load(const unsigned char *row, int sw, int kk, int half) {
        const i32x4 a = *reinterpret_cast<const i32x4 *>(row + ((kk * 4 + half) ^ sw) * 16);
        const i32x4 b = *reinterpret_cast<const i32x4 *>(row + ((kk * 4 + 2 + half) ^ sw) * 16);
        return (i32x8){a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    }
    // the block scales are 2^(127 - 127) = 1
    __device__ static __forceinline__ f16v mfma(i32x8 a, i32x8 b, f16v c) {
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 0x7f7f7f7f, 0, 0x7f7f7f7f);
    }
};

// KTAIL: K is no whole number of steps, so each load checks its chunk; otherwise the
// K position rides in the scalar offset and the per-lane offsets are fixed.
template <class S, bool FP8, bool KTAIL>
__global__ __launch_bounds__(64 * S::NW, S::NW * S::PER_CU / 4) void linear_kernel(Args g) {
    using F = Frag<FP8>;
    using frag = typename F::type;
    constexpr int FI = S::FI, TJ = S::TJ, KK = kStep / F::BYTES, LA = S::LA, LB = S::LB, SA = S::SA, SB = S::SB;
    static_assert(KK % 2 == 0, "a step's first sub-step is always in the first fragment set");
    __shared__ __attribute__((aligned(1024))) unsigned char lds[S::LDS];

    // Workgroups are dealt round robin over the 8 XCDs; each XCD walks a contiguous range of the
    // tile order: groups of four token tiles, feature tiles within a group, its token tiles fastest,
    // so the tiles an XCD runs at once share their operands in its L2; the K splits are outermost.
    const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
    const int tile = xcd * g.per_xcd + slot;
    const int tiles = g.tiles_f * g.tiles_t;
    if (slot >= g.per_xcd || tile >= tiles * g.splits) return;
    const int ks = tile / tiles, mn = tile - ks * tiles;
    constexpr int GROUP = 4;
    const int first_t = mn / (GROUP * g.tiles_f) * GROUP;
    const int gt = min(GROUP, g.tiles_t - first_t);
    const int within = mn - first_t * g.tiles_f;
    const int t0 = (first_t + within % gt) * S::BT, f0 = within / gt * S::BF;
    const int steps_total = (g.kbytes + kStep - 1) / kStep;
    const int kbeg = static_cast<int>(static_cast<int64_t>(steps_total) * ks / g.splits);
    const int kend = static_cast<int>(static_cast<int64_t>(steps_total) * (ks + 1) / g.splits);
    const int nsteps = kend - kbeg;

    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wf = wave / S::WT, wt = wave % S::WT;
    // the descriptors end with the tile's last valid row, so rows past M or n read as zeros
    const int fr = min(S::BF, g.M - f0), tr = min(S::BT, g.n - t0);
    const __amdgpu_buffer_rsrc_t rsA = uniform_rsrc(
        g.w + static_cast<int64_t>(f0) * g.ldw, static_cast<uint32_t>((fr - 1) * g.ldw + g.kbytes));
    const __amdgpu_buffer_rsrc_t rsB = uniform_rsrc(
        g.x + static_cast<int64_t>(t0) * g.ldx, static_cast<uint32_t>((tr - 1) * g.ldx + g.kbytes));

    // this wave's loads: kLoadRows rows of kStep bytes each, lane -> row lane / kChunks, position lane % kChunks
    constexpr int kMaxLoads = 8;
    static_assert(LA <= kMaxLoads && LB <= kMaxLoads, "load slots");
    uint32_t voffA[kMaxLoads], voffB[kMaxLoads];
    const int lrow = lane / kChunks, lpos = lane % kChunks;
    // byte of K the lane's chunk starts at: load blocks alternate between two
    int kb[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) kb[p] = (lpos ^ swz(p * kLoadRows + lrow)) * 16;
#pragma unroll
    for (int j = 0; j < LA; ++j) {
        const int r = (j * S::NW + wave) * kLoadRows + lrow;
        voffA[j] = static_cast<uint32_t>(r) * static_cast<uint32_t>(g.ldw) + (lpos ^ swz(r)) * 16u;
    }
#pragma unroll
    for (int j = 0; j < LB; ++j) {
        const int r = (j * S::NW + wave) * kLoadRows + lrow;
        voffB[j] = static_cast<uint32_t>(r) * static_cast<uint32_t>(g.ldx) + (lpos ^ swz(r)) * 16u;
    }
    auto load_a = [&](int step, int slot_a) {
#pragma unroll
        for (int j = 0; j < LA; ++j) {
            unsigned char *dst = lds + slot_a * S::A_BYTES + (j * S::NW + wave) * 1024;
            const int k0 = step * kStep;
            if constexpr (KTAIL) {
                const uint32_t v = k0 + kb[(j * S::NW + wave) & 1] >= g.kbytes ? kOutside : voffA[j] + k0;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsA, (lds_ptr)dst, 16, v, 0, 0, 0);
            } else {
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsA, (lds_ptr)dst, 16, voffA[j], k0, 0, 0);
            }
        }
    };
    auto load_b = [&](int step, int slot_b) {
#pragma unroll
        for (int j = 0; j < LB; ++j) {
            unsigned char *dst = lds + SA * S::A_BYTES + slot_b * S::B_BYTES + (j * S::NW + wave) * 1024;
            const int k0 = step * kStep;
            if constexpr (KTAIL) {
                const uint32_t v = k0 + kb[(j * S::NW + wave) & 1] >= g.kbytes ? kOutside : voffB[j] + k0;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsB, (lds_ptr)dst, 16, v, 0, 0, 0);
            } else {
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsB, (lds_ptr)dst, 16, voffB[j], k0, 0, 0);
            }
        }
    };
    auto read_frags = [&](int slot_a, int slot_b, int kk, frag *af, frag *bf) {
        const unsigned char *At = lds + slot_a * S::A_BYTES, *Bt = lds + SA * S::A_BYTES + slot_b * S::B_BYTES;
#pragma unroll
        for (int i = 0; i < FI; ++i) {
            const int r = (wf * FI + i) * 32 + (lane & 31);
            af[i] = F::load(At + r * kStep, swz(r), kk, half);
        }
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            const int r = (wt * TJ + j) * 32 + (lane & 31);
            bf[j] = F::load(Bt + r * kStep, swz(r), kk, half);
        }
    };
    // Spread the next sub-step's LDS reads, and in sub-step 0 the loads, between the MFMAs.
    auto interleave = [&](int kk) {
        constexpr int NM = FI * TJ, NR = (FI + TJ) * (FP8 ? 2 : 1), NS = NM > 2 ? NM - 2 : NM;
        if constexpr (NM >= 4) {
#pragma unroll
            for (int q = 0; q < NM; ++q) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                       // MFMA
                const int nr = q < NS ? NR / NS + (q < NR % NS ? 1 : 0) : 0;
                if (nr == 4) __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);          // LDS reads
                else if (nr == 3) __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
                else if (nr == 2) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
                else if (nr == 1) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                if (kk == 0 && q < LA + LB) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);   // VMEM read
            }
        }
    };

    f16v acc[FI][TJ];
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = (f16v){};
    frag a0[FI], b0[TJ], a1[FI], b1[TJ];

    // Order of requests: x of step s + SB - 1, then w of step s + SA - 1, at the start of step s.  When
    // step s ends, this many of the wave's newest loads may be outstanding while step s + 1 is whole.
    constexpr int LEFT = (SB - 2) * (LA + LB) + (SA > SB ? LA : 0);
    static_assert(LEFT < 64, "vmcnt");
    if (nsteps > 0) {
        // as steps before 0 would have asked for them
        for (int s = 1 - SA; s < 0; ++s) {
            const int tb = s + SB - 1, ta = s + SA - 1;
            if (tb >= 0 && tb < nsteps) load_b(kbeg + tb, tb % SB);
            if (ta < nsteps) load_a(kbeg + ta, ta % SA);
        }
        if (nsteps >= SA) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LEFT) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        asm volatile("s_barrier" ::: "memory");
        read_frags(0, 0, 0, a0, b0);
    }
    // settle the scalar loads so the LDS waits inside the loop count precisely
    __builtin_amdgcn_s_waitcnt(0xC07F);
    int sa = 0, sb = 0;   // slots of step s
    auto one_step = [&](int s) {
        const int na = sa + 1 == SA ? 0 : sa + 1, nb = sb + 1 == SB ? 0 : sb + 1;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            const bool odd = kk & 1;
            frag *ac = odd ? a1 : a0, *bc = odd ? b1 : b0;
            frag *an = odd ? a0 : a1, *bn = odd ? b0 : b1;
            __builtin_amdgcn_sched_barrier(0);
            if (kk == 0) {
                // the slots before these were read in step s - 1, which every wave ended at the barrier
                if (s + SB - 1 < nsteps) load_b(kbeg + s + SB - 1, sb == 0 ? SB - 1 : sb - 1);
                if (s + SA - 1 < nsteps) load_a(kbeg + s + SA - 1, sa == 0 ? SA - 1 : sa - 1);
            }
            if (kk + 1 < KK) {
                read_frags(sa, sb, kk + 1, an, bn);
            } else {
                // this wave's fragments are in registers and its loads of step s + 1 have landed; after
                // the barrier so are everyone's.  (After the last step this reads a tile again, unused.)
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                if (s + SA - 1 < nsteps) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LEFT) : "memory");
                else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                asm volatile("s_barrier" ::: "memory");
                read_frags(na, nb, 0, an, bn);
            }
#pragma unroll
            for (int i = 0; i < FI; ++i)
#pragma unroll
                for (int j = 0; j < TJ; ++j) acc[i][j] = F::mfma(ac[i], bc[j], acc[i][j]);
            interleave(kk);
        }
        sa = na;
        sb = nb;
    };
    for (int s = 0; s < nsteps; ++s) one_step(s);

    // epilogue: a wave's own LDS region, 32 tokens at a time
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __syncthreads();   // every wave is done with the operand tiles
    constexpr int LPT = FI * 4, TPP = 64 / LPT;   // lanes per token, tokens per pass
    constexpr int PASSES = 32 / TPP, U = PASSES < 4 ? PASSES : 4;
    float *reg = reinterpret_cast<float *>(lds) + wave * 32 * S::OUT_LD;
    const int lf = (lane % LPT) * 8;
    const int64_t f = f0 + wf * FI * 32 + lf;
    const bool split = g.splits > 1;
    Cols cols;
    if (!split) cols = load_cols(g.e, f);
    // a lane's accumulators belong to one token per j: its scale goes in here
    float sx[TJ];
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
        const int64_t t = t0 + (wt * TJ + j) * 32 + (lane & 31);
        sx[j] = FP8 && g.e.scale_x && t < g.n ? g.e.scale_x[t] : 1.0f;
    }
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
#pragma unroll
        for (int i = 0; i < FI; ++i)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                float4 q = make_float4(acc[i][j][r], acc[i][j][r + 1], acc[i][j][r + 2], acc[i][j][r + 3]);
                if constexpr (FP8) {
                    q.x *= sx[j];
                    q.y *= sx[j];
                    q.z *= sx[j];
                    q.w *= sx[j];
                }
                *reinterpret_cast<float4 *>(reg + (lane & 31) * S::OUT_LD + i * 32 + (r >> 2) * 8 + half * 4) = q;
            }
        __builtin_amdgcn_wave_barrier();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll 1   // the accumulators are in LDS: one copy of the epilogue per j
        for (int p0 = 0; p0 < PASSES; p0 += U) {
            const int tl = p0 * TPP + lane / LPT;
            const int64_t t = t0 + (wt * TJ + j) * 32 + tl;
            auto read = [&](float (&v)[U][8]) {
#pragma unroll
                for (int p = 0; p < U; ++p) {
                    const float4 x = *reinterpret_cast<const float4 *>(reg + (tl + p * TPP) * S::OUT_LD + lf);
                    const float4 y = *reinterpret_cast<const float4 *>(reg + (tl + p * TPP) * S::OUT_LD + lf + 4);
                    v[p][0] = x.x; v[p][1] = x.y; v[p][2] = x.z; v[p][3] = x.w;
                    v[p][4] = y.x; v[p][5] = y.y; v[p][6] = y.z; v[p][7] = y.w;
                }
            };
            if (f >= g.M) continue;
            if (!split) {
                finish<U>(g.e, cols, t, TPP, f, read);
            } else {   // ldpart is M in whole eights
                float v[U][8];
                read(v);
#pragma unroll
                for (int p = 0; p < U; ++p) {
                    if (t + p * TPP >= g.n) continue;
                    float4 *o = reinterpret_cast<float4 *>(
                        g.part + (static_cast<int64_t>(ks) * g.n + t + p * TPP) * g.ldpart + f);
                    o[0] = make_float4(v[p][0], v[p][1], v[p][2], v[p][3]);
                    o[1] = make_float4(v[p][4], v[p][5], v[p][6], v[p][7]);
                }
            }
        }
        __builtin_amdgcn_wave_barrier();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// The partial sums of the K splits, added in their order, through the epilogue.
__global__ __launch_bounds__(256) inline void linear_fold_kernel(const float *part, int64_t ldpart, int splits, Epi e) {
    const int64_t per = ldpart / 8, total = e.n * per;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t t = i / per, f = (i - t * per) * 8;
        const float *p = part + t * ldpart + f;
        float4 u = reinterpret_cast<const float4 *>(p)[0], v = reinterpret_cast<const float4 *>(p)[1];
        for (int k = 1; k < splits; ++k) {
            const float4 *q = reinterpret_cast<const float4 *>(p + static_cast<int64_t>(k) * e.n * ldpart);
            const float4 a = q[0], b = q[1];
            u.x += a.x; u.y += a.y; u.z += a.z; u.w += a.w;
            v.x += b.x; v.y += b.y; v.z += b.z; v.w += b.w;
        }
        const Cols c = load_cols(e, f);
        finish<1>(e, c, t, 0, f, [&](float (&s)[1][8]) {
            s[0][0] = u.x; s[0][1] = u.y; s[0][2] = u.z; s[0][3] = u.w;
            s[0][4] = v.x; s[0][5] = v.y; s[0][6] = v.z; s[0][7] = v.w;
        });
    }
}

// ---- few tokens ------------------------------------------------------------------------
//
// Up to 32 tokens: the weight is read once and little else happens, so the time is how soon and how
// widely its reads go out.  A workgroup takes 16 features and its eight waves an eighth of K each, so
// a 4096 x 4096 weight already keeps 2048 waves reading without splitting K over workgroups (whose
// partial sums and second launch cost 3 us of 11: 4 x 4640 x 1880 e4m3 takes 6.7 us here, 12.2 split).  Operands go straight from memory to the MFMA's
// registers: lane l supplies row l % 16 of w (token l % 16 of x) and the 16-byte chunk l / 16 of every
// 64 bytes of K, eight (or with two token tiles four) such loads ahead of those in use.  The waves'
// sums meet in LDS, are added in wave order and go through the epilogue one value per lane.
constexpr int kRowsWaves = 8;

template <bool FP8>
__device__ __forceinline__ void mfma16(f4v &acc, const u32x4 &a, const u32x4 &b) {
    if constexpr (FP8) {   // 16 bytes are two 8-byte operands
        acc = __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(
            static_cast<long>((static_cast<uint64_t>(a.y) << 32) | a.x),
            static_cast<long>((static_cast<uint64_t>(b.y) << 32) | b.x), acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(
            static_cast<long>((static_cast<uint64_t>(a.w) << 32) | a.z),
            static_cast<long>((static_cast<uint64_t>(b.w) << 32) | b.z), acc, 0, 0, 0);
    } else {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), acc, 0, 0, 0);
    }
}

template <bool FP8, int TT>   // token tiles of 16
__global__ __launch_bounds__(64 * kRowsWaves, 2) void linear_rows_kernel(Args g) {
    constexpr int U = TT == 1 ? 8 : 4;   // loads of w at once
    __shared__ __attribute__((aligned(16))) float sums[kRowsWaves][TT * 256];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int f0 = blockIdx.x * 16;
    const int rows = min(16, g.M - f0);
    const __amdgpu_buffer_rsrc_t rsW = uniform_rsrc(
        g.w + static_cast<int64_t>(f0) * g.ldw, static_cast<uint32_t>((rows - 1) * g.ldw + g.kbytes));
    const __amdgpu_buffer_rsrc_t rsX = uniform_rsrc(g.x, static_cast<uint32_t>((g.n - 1) * g.ldx + g.kbytes));
    const int chunk = (lane >> 4) * 16;   // byte of the lane's chunk in every 64
    const uint32_t vw = static_cast<uint32_t>(lane & 15) * static_cast<uint32_t>(g.ldw) + chunk;
    uint32_t vx[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t)
        vx[t] = static_cast<uint32_t>(t * 16 + (lane & 15)) * static_cast<uint32_t>(g.ldx) + chunk;
    const int total = (g.kbytes + 63) / 64;
    const int beg = static_cast<int>(static_cast<int64_t>(total) * wave / kRowsWaves);
    const int end = static_cast<int>(static_cast<int64_t>(total) * (wave + 1) / kRowsWaves);
    auto fetch = [&](int s, u32x4 (&w)[U], u32x4 (&x)[TT][U]) {   // zeros past this wave's share and past K
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = s + u < end && (s + u) * 64 + chunk < g.kbytes;
            const uint32_t k = static_cast<uint32_t>(s + u) * 64u;
            w[u] = __builtin_amdgcn_raw_buffer_load_b128(rsW, in ? vw + k : kOutside, 0, 0);
#pragma unroll
            for (int t = 0; t < TT; ++t) x[t][u] = __builtin_amdgcn_raw_buffer_load_b128(rsX, in ? vx[t] + k : kOutside, 0, 0);
        }
    };
    f4v acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = (f4v){0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 w0[U], w1[U], x0[TT][U], x1[TT][U];
    auto use = [&](u32x4 (&w)[U], u32x4 (&x)[TT][U]) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int t = 0; t < TT; ++t) mfma16<FP8>(acc[t], w[u], x[t][u]);
    };
    fetch(beg, w0, x0);
    for (int s = beg; s < end; s += 2 * U) {
        fetch(s + U, w1, x1);
        use(w0, x0);
        fetch(s + 2 * U, w0, x0);
        use(w1, x1);
    }
    // result register r of lane l: feature (l / 16) 4 + r, token l % 16
#pragma unroll
    for (int t = 0; t < TT; ++t)
        *reinterpret_cast<f4v *>(&sums[wave][t * 256 + (lane & 15) * 16 + (lane >> 4) * 4]) = acc[t];
    __syncthreads();
    const Epi &e = g.e;
    const int i = threadIdx.x;
    if (i >= TT * 256) return;
    const int64_t t = i >> 4, f = f0 + (i & 15);
    if (t >= e.n || f >= e.M) return;
    float v = sums[0][i];
#pragma unroll
    for (int k = 1; k < kRowsWaves; ++k) v += sums[k][i];
    if (FP8 && e.scale_x) v *= e.scale_x[t];
    if (FP8 && e.scale_w) v *= e.scale_w[f];
    if (e.bias) v += e.bias_bf16 ? Elt<true>::load_one(e.bias, f) : static_cast<const float *>(e.bias)[f];
    if (e.preact) Elt<true>::store_one(e.preact, t * e.ldp + f, v);
    v = activate(e.act, v);
    if (e.out_bf16) {
        if (e.residual) v += Elt<true>::load_one(e.residual, t * e.ldr + f);
        Elt<true>::store_one(e.out, t * e.ldo + f, v);
    } else {
        if (e.residual) v += static_cast<const float *>(e.residual)[t * e.ldr + f];
        static_cast<float *>(e.out)[t * e.ldo + f] = v;
    }
}

}  // namespace linear
}  // namespace lce
