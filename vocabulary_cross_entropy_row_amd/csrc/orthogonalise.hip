// Orthogonalised update by Newton-Schulz products, over X = G / (||G||_F + eps) with r rows and c >= r
// columns (G transposed if it is taller than wide), `steps` times:
//   A = X X^T,   B = b A + c A A,   X <- a X + B X
//
// The three products run on the matrix cores in fp16, whose 11 bits keep eight times what bf16 does at the
// same rate, with fp32 sums.  What would be lost is kept where it costs nothing:
//   X      two fp16, hi + lo: the products read hi, the term a X both.  The products' share of X is small
//          in the directions that a X still has to amplify, so those see no rounding of X.
//   A, B   their diagonals in fp32 vectors, the rest in fp16.  X approaches orthogonal rows, so A
//          approaches its diagonal: A = D + O gives A A = O O + (D_t + D_f) O + D^2, and B X = diag X + rest.
// Simulated over gaussian, low-rank and power-law spectra (256 to 1024 rows): 2e-4 to 7e-4 of the result
// (2-norm) where fp16 alone gives 1e-3 to 4e-3 and bf16 1e-2 to 3e-2; the bf16 output rounds at 1.7e-3.
// Powers of two keep fp16 in range: X is held times S ~ sqrt(c) (|X| is at most about 1.2, its root mean
// square at most 1.2 / sqrt(c)), O times 2^10, B times 2^8.
//
// A and A A are symmetric: only tiles on and below the diagonal are computed, and stored a second time
// transposed.  All operands have K contiguous: X for A, O for O O, and for B X also X^T (hi), which the
// product that forms X writes beside it.  A step is three launches, r^2 c + r^3 + 2 r^2 c operations.
// Everything is padded with zeros to multiples of 64, so the products meet no edges.
#include <hip/hip_runtime.h>
#include <algorithm>
#include <math.h>
#include <stdint.h>

#include "blocks_internal.h"
#include "ce_device.h"
#include "linear_mfma.h"

namespace lce {
namespace {

using dev::Elt;
using dev::u32x4;
using linear::any16;
using linear::f16v;
using linear::kChunks;
using linear::kLoadRows;
using linear::kStep;
using linear::lds_ptr;
using linear::swz;
using linear::uniform_rsrc;

typedef _Float16 h8 __attribute__((ext_vector_type(8)));

constexpr int64_t kUnit = 64;             // fp16 values of K in a step
constexpr float kScaleO = 1024.0f, kScaleB = 256.0f;
constexpr int kNormGroups = 64;           // partial sums of squares per matrix

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }
size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

__device__ __forceinline__ u32x4 pack_h8(const float (&v)[8]) {
    h8 h;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = static_cast<_Float16>(v[e]);
    return __builtin_bit_cast(u32x4, h);
}

// ---- the norm, and X in fp16 -----------------------------------------------------------------

struct LoadArgs {
    const void *g;
    int64_t ldg, gb;                  // strides of G (elements)
    int64_t rows, cols;               // of G
    double *part;                     // [batch][kNormGroups]
    uint16_t *hi, *lo, *xt;           // X [rp][ldx], X^T [cp][ldt]
    int64_t ldx, ldt, xb, tb;         // row and batch strides (elements)
    int rp, cp;                       // padded rows and columns of X
    int tall;                         // X is G^T
    float s, eps;
};

// Sums of squares in fp64, a fixed share of the rows' 1024-value pieces per workgroup: no square of a
// finite fp32 value overflows, and the order is fixed.
template <bool BF16>
__global__ __launch_bounds__(256) void norm_kernel(LoadArgs a) {
    __shared__ double sums[4];
    const int64_t pieces = (a.cols + 1023) / 1024, total = a.rows * pieces;
    const int64_t base = blockIdx.y * a.gb;
    double sum = 0.0;
    for (int64_t i = blockIdx.x; i < total; i += kNormGroups) {
        const int64_t row = i / pieces, c = (i - row * pieces) * 1024 + threadIdx.x * 4;
        const int64_t at = base + row * a.ldg + c;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = c + e < a.cols ? Elt<BF16>::load_one(a.g, at + e) : 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += static_cast<double>(v[e]) * static_cast<double>(v[e]);
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) a.part[blockIdx.y * kNormGroups + blockIdx.x] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// A workgroup takes 64 x 64 of X: hi, lo and the transposed hi, zeros in the padding.
template <bool BF16>
__global__ __launch_bounds__(256) void load_kernel(LoadArgs a) {
    __shared__ float tile[64][65];
    __shared__ float factor;
    const int t = threadIdx.x, z = blockIdx.z;
    if (t < 64) {
        double s = a.part[z * kNormGroups + t];
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) s += __shfl_xor(s, m);
        if (t == 0) factor = static_cast<float>(static_cast<double>(a.s) / (sqrt(s) + static_cast<double>(a.eps)));
    }
    const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;   // of X
    const int g0 = a.tall ? c0 : r0, h0 = a.tall ? r0 : c0;   // of G
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int64_t row = g0 + i * 4 + (t >> 6), col = h0 + (t & 63);
        v[i] = row < a.rows && col < a.cols ? Elt<BF16>::load_one(a.g, z * a.gb + row * a.ldg + col) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) tile[i * 4 + (t >> 6)][t & 63] = v[i] * factor;
    __syncthreads();
    // eight values along a row of X, and along a row of X^T
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int line = i * 32 + (t >> 3), at = (t & 7) * 8;
        float p[8], q[8], rest[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            p[e] = tile[line][at + e];   // of G
            q[e] = tile[at + e][line];
        }
        if (a.tall) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = p[e];
                p[e] = q[e];
                q[e] = x;
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) rest[e] = p[e] - static_cast<float>(static_cast<_Float16>(p[e]));
        const int64_t x_at = z * a.xb + static_cast<int64_t>(r0 + line) * a.ldx + c0 + at;
        *reinterpret_cast<u32x4 *>(a.hi + x_at) = pack_h8(p);
        *reinterpret_cast<u32x4 *>(a.lo + x_at) = pack_h8(rest);
        *reinterpret_cast<u32x4 *>(a.xt + z * a.tb + static_cast<int64_t>(c0 + line) * a.ldt + r0 + at) = pack_h8(q);
    }
}

// ---- products ----------------------------------------------------------------------------------

enum { GRAM, POLY, APPLY, LAST };

struct Args {
    const uint16_t *w, *x;            // K contiguous: features [rows_w][ldw], tokens [rows_x][ldx]
    int64_t ldw, ldx, wb, xb;         // row and batch strides (elements)
    int rows_w, rows_x;               // multiples of 64
    int steps;                        // of K
    int tiles_f, per_batch, total, splits, per_xcd;   // tiles; per_batch: of one matrix, all splits
    float *part;                      // splits > 1: [batch][splits][rows][rows] fp32
    // epilogue
    float inv;                        // of the products' scale
    uint16_t *o;                      // O [rows][ldo]: written by GRAM, read by POLY
    uint16_t *bo;                     // B's off-diagonal part
    int64_t ldo, ob;
    float *d, *e;                     // diagonals of A, and a + that of B: [batch][rows]
    float a, b, c;
    uint16_t *hi, *lo, *xt;           // X and the next X^T
    int64_t ldh, hb, ldt, tb;
    void *out;                        // LAST: bf16
    int64_t ldout, outb;
    int64_t r, cols;                  // of X, not padded
    int tall;
};

// GRAM: values v of A to O and its diagonal.  POLY: values of O O to B.
template <int EPI>
__device__ __forceinline__ void symmetric_values(const Args &g, int z, int t, int f, float (&v)[8]) {
    float *d = g.d + static_cast<int64_t>(z) * g.rows_x;
    if constexpr (EPI == GRAM) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            v[u] *= g.inv;
            if (t == f + u) {
                d[t] = v[u];
                v[u] = 0.0f;
            }
            v[u] *= kScaleO;
        }
    } else {
        const u32x4 oq = *reinterpret_cast<const u32x4 *>(g.o + z * g.ob + static_cast<int64_t>(t) * g.ldo + f);
        const h8 o = __builtin_bit_cast(h8, oq);
        const float dt = d[t];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const float df = d[f + u], ov = static_cast<float>(o[u]) * (1.0f / kScaleO);
            float square = fmaf(dt + df, ov, v[u] * g.inv);
            if (t == f + u) {
                square = fmaf(dt, dt, square);   // O is 0 there
                g.e[static_cast<int64_t>(z) * g.rows_x + t] = g.a + fmaf(g.c, square, g.b * dt);
                v[u] = 0.0f;
            } else {
                v[u] = fmaf(g.c, square, g.b * ov) * kScaleB;
            }
        }
    }
}

template <class S, int EPI>
__global__ __launch_bounds__(64 * S::NW, S::NW * S::PER_CU / 4) void ortho_kernel(Args g) {
    constexpr int FI = S::FI, TJ = S::TJ, KK = 4, LA = S::LA, LB = S::LB, SA = S::SA, SB = S::SB;
    constexpr bool SYM = EPI == GRAM || EPI == POLY;
    static_assert(!SYM || S::BF == S::BT, "tiles of a symmetric product are square");
    __shared__ __attribute__((aligned(1024))) unsigned char lds[S::LDS];

    // each XCD walks a contiguous range of the tiles
    const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
    const int tile = xcd * g.per_xcd + slot;
    if (slot >= g.per_xcd || tile >= g.total) return;
    const int z = tile / g.per_batch, in_batch = tile - z * g.per_batch;
    const int per_split = g.per_batch / g.splits, ks = in_batch / per_split, mn = in_batch - ks * per_split;
    int ti, fi;
    if constexpr (SYM) {   // row ti of the lower triangle holds ti + 1 tiles
        ti = static_cast<int>((sqrtf(8.0f * static_cast<float>(mn) + 1.0f) - 1.0f) * 0.5f);
        while (ti * (ti + 1) / 2 > mn) --ti;
        while ((ti + 1) * (ti + 2) / 2 <= mn) ++ti;
        fi = mn - ti * (ti + 1) / 2;
    } else {   // groups of four token tiles, its token tiles fastest
        constexpr int GROUP = 4;
        const int tiles_t = per_split / g.tiles_f;
        const int first_t = mn / (GROUP * g.tiles_f) * GROUP;
        const int gt = min(GROUP, tiles_t - first_t);
        const int within = mn - first_t * g.tiles_f;
        ti = first_t + within % gt;
        fi = within / gt;
    }
    const int t0 = ti * S::BT, f0 = fi * S::BF;
    const int kbeg = static_cast<int>(static_cast<int64_t>(g.steps) * ks / g.splits);
    const int nsteps = static_cast<int>(static_cast<int64_t>(g.steps) * (ks + 1) / g.splits) - kbeg;

    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wf = wave / S::WT, wt = wave % S::WT;
    const int fr = min(S::BF, g.rows_w - f0), tr = min(S::BT, g.rows_x - t0);
    const uint32_t ldw = static_cast<uint32_t>(g.ldw * 2), ldx = static_cast<uint32_t>(g.ldx * 2), kbytes = g.steps * kStep;
    const __amdgpu_buffer_rsrc_t rsA = uniform_rsrc(g.w + z * g.wb + f0 * g.ldw, (fr - 1) * ldw + kbytes);
    const __amdgpu_buffer_rsrc_t rsB = uniform_rsrc(g.x + z * g.xb + t0 * g.ldx, (tr - 1) * ldx + kbytes);
    constexpr int kMaxLoads = 8;
    static_assert(LA <= kMaxLoads && LB <= kMaxLoads, "load slots");
    uint32_t voffA[kMaxLoads], voffB[kMaxLoads];
    const int lrow = lane / kChunks, lpos = lane % kChunks;
#pragma unroll
    for (int j = 0; j < LA; ++j) {
        const int r = (j * S::NW + wave) * kLoadRows + lrow;
        voffA[j] = static_cast<uint32_t>(r) * ldw + (lpos ^ swz(r)) * 16u;
    }
#pragma unroll
    for (int j = 0; j < LB; ++j) {
        const int r = (j * S::NW + wave) * kLoadRows + lrow;
        voffB[j] = static_cast<uint32_t>(r) * ldx + (lpos ^ swz(r)) * 16u;
    }
    auto load_a = [&](int step, int slot_a) {
#pragma unroll
        for (int j = 0; j < LA; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsA, (lds_ptr)(lds + slot_a * S::A_BYTES + (j * S::NW + wave) * 1024), 16,
                                                     voffA[j], step * kStep, 0, 0);
    };
    auto load_b = [&](int step, int slot_b) {
#pragma unroll
        for (int j = 0; j < LB; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsB, (lds_ptr)(lds + SA * S::A_BYTES + slot_b * S::B_BYTES + (j * S::NW + wave) * 1024), 16, voffB[j],
                step * kStep, 0, 0);
    };
    auto read_frags = [&](int slot_a, int slot_b, int kk, h8 *af, h8 *bf) {
        const unsigned char *At = lds + slot_a * S::A_BYTES, *Bt = lds + SA * S::A_BYTES + slot_b * S::B_BYTES;
#pragma unroll
        for (int i = 0; i < FI; ++i) {
            const int r = (wf * FI + i) * 32 + (lane & 31);
            af[i] = *reinterpret_cast<const h8 *>(At + r * kStep + ((kk * 2 + half) ^ swz(r)) * 16);
        }
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            const int r = (wt * TJ + j) * 32 + (lane & 31);
            bf[j] = *reinterpret_cast<const h8 *>(Bt + r * kStep + ((kk * 2 + half) ^ swz(r)) * 16);
        }
    };
    // Spread the next sub-step's LDS reads, and in sub-step 0 the loads, between the MFMAs.
    auto interleave = [&](int kk) {
        constexpr int NM = FI * TJ, NR = FI + TJ, NS = NM > 2 ? NM - 2 : NM;
        if constexpr (NM >= 4) {
#pragma unroll
            for (int q = 0; q < NM; ++q) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                       // MFMA
                const int nr = q < NS ? NR / NS + (q < NR % NS ? 1 : 0) : 0;
                if (nr == 2) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);          // LDS reads
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
    h8 a0[FI], b0[TJ], a1[FI], b1[TJ];
    // The order of requests, and how many may be outstanding when a step ends, are linear_kernel's.
    constexpr int LEFT = (SB - 2) * (LA + LB) + (SA > SB ? LA : 0);
    static_assert(LEFT < 64, "vmcnt");
    for (int s = 1 - SA; s < 0; ++s) {
        const int tb = s + SB - 1, ta = s + SA - 1;
        if (tb >= 0 && tb < nsteps) load_b(kbeg + tb, tb % SB);
        if (ta < nsteps) load_a(kbeg + ta, ta % SA);
    }
    if (nsteps >= SA) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LEFT) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    asm volatile("s_barrier" ::: "memory");
    read_frags(0, 0, 0, a0, b0);
    __builtin_amdgcn_s_waitcnt(0xC07F);
    int sa = 0, sb = 0;
    auto one_step = [&](int s) {
        const int na = sa + 1 == SA ? 0 : sa + 1, nb = sb + 1 == SB ? 0 : sb + 1;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            const bool odd = kk & 1;
            h8 *ac = odd ? a1 : a0, *bc = odd ? b1 : b0;
            h8 *an = odd ? a0 : a1, *bn = odd ? b0 : b1;
            __builtin_amdgcn_sched_barrier(0);
            if (kk == 0) {
                if (s + SB - 1 < nsteps) load_b(kbeg + s + SB - 1, sb == 0 ? SB - 1 : sb - 1);
                if (s + SA - 1 < nsteps) load_a(kbeg + s + SA - 1, sa == 0 ? SA - 1 : sa - 1);
            }
            if (kk + 1 < KK) {
                read_frags(sa, sb, kk + 1, an, bn);
            } else {
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                if (s + SA - 1 < nsteps) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LEFT) : "memory");
                else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                asm volatile("s_barrier" ::: "memory");
                read_frags(na, nb, 0, an, bn);
            }
#pragma unroll
            for (int i = 0; i < FI; ++i)
#pragma unroll
                for (int j = 0; j < TJ; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ac[i], bc[j], acc[i][j], 0, 0, 0);
            interleave(kk);
        }
        sa = na;
        sb = nb;
    };
    for (int s = 0; s < nsteps; ++s) one_step(s);

    // epilogue: a wave's own LDS region, 32 tokens at a time, eight features of a token per lane
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __syncthreads();
    constexpr int LPT = FI * 4, TPP = 64 / LPT, PASSES = 32 / TPP;
    float *reg = reinterpret_cast<float *>(lds) + wave * 32 * S::OUT_LD;
    const int lf = (lane % LPT) * 8;
    const int f = f0 + wf * FI * 32 + lf;
    // rows of X^T, of the mirrored tile, or of the output of a tall matrix
    const bool turned = EPI == APPLY || (SYM && ti != fi && g.splits == 1) || (EPI == LAST && g.tall);
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
        const int tj = t0 + (wt * TJ + j) * 32;
#pragma unroll
        for (int i = 0; i < FI; ++i)
#pragma unroll
            for (int r = 0; r < 16; r += 4)
                *reinterpret_cast<float4 *>(reg + (lane & 31) * S::OUT_LD + i * 32 + (r >> 2) * 8 + half * 4) =
                    make_float4(acc[i][j][r], acc[i][j][r + 1], acc[i][j][r + 2], acc[i][j][r + 3]);
        __builtin_amdgcn_wave_barrier();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (tj >= g.rows_x || f0 + wf * FI * 32 >= g.rows_w) continue;   // rows come in 64s: all 32, and all or none of each 32 features
#pragma unroll 2
        for (int p = 0; p < PASSES; ++p) {
            const int tl = p * TPP + lane / LPT, t = tj + tl;
            float *at = reg + tl * S::OUT_LD + lf;
            if (f >= g.rows_w) continue;
            const float4 x = reinterpret_cast<const float4 *>(at)[0], y = reinterpret_cast<const float4 *>(at)[1];
            float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
            if constexpr (SYM) {
                if (g.splits > 1) {
                    float4 *o = reinterpret_cast<float4 *>(
                        g.part + ((static_cast<int64_t>(z) * g.splits + ks) * g.rows_x + t) * g.rows_x + f);
                    o[0] = x;
                    o[1] = y;
                    continue;
                }
                symmetric_values<EPI>(g, z, t, f, v);
                *reinterpret_cast<u32x4 *>((EPI == GRAM ? g.o : g.bo) + z * g.ob + static_cast<int64_t>(t) * g.ldo + f) = pack_h8(v);
            } else {
                const int64_t h_at = z * g.hb + static_cast<int64_t>(t) * g.ldh + f;
                const h8 hi = __builtin_bit_cast(h8, *reinterpret_cast<const u32x4 *>(g.hi + h_at));
                const h8 lo = __builtin_bit_cast(h8, *reinterpret_cast<const u32x4 *>(g.lo + h_at));
                const float e = g.e[static_cast<int64_t>(z) * g.rows_x + t];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    v[u] = fmaf(e, static_cast<float>(hi[u]) + static_cast<float>(lo[u]), v[u] * (1.0f / kScaleB));
                if constexpr (EPI == APPLY) {
                    float rest[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) rest[u] = v[u] - static_cast<float>(static_cast<_Float16>(v[u]));
                    *reinterpret_cast<u32x4 *>(g.hi + h_at) = pack_h8(v);
                    *reinterpret_cast<u32x4 *>(g.lo + h_at) = pack_h8(rest);
                } else {
#pragma unroll
                    for (int u = 0; u < 8; ++u) v[u] *= g.inv;
                    if (!g.tall && t < g.r) {
                        uint16_t *o = static_cast<uint16_t *>(g.out) + z * g.outb + static_cast<int64_t>(t) * g.ldout + f;
                        if (f + 8 <= g.cols) {
                            *reinterpret_cast<any16 *>(o) = Elt<true>::pack(v);
                        } else {
#pragma unroll
                            for (int u = 0; u < 8; ++u)
                                if (f + u < g.cols) Elt<true>::store_one(o, u, v[u]);
                        }
                    }
                }
            }
            if (turned) {
                reinterpret_cast<float4 *>(at)[0] = make_float4(v[0], v[1], v[2], v[3]);
                reinterpret_cast<float4 *>(at)[1] = make_float4(v[4], v[5], v[6], v[7]);
            }
        }
        __builtin_amdgcn_wave_barrier();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (turned) {   // four lanes a feature, eight of its 32 tokens each
#pragma unroll 2
            for (int q = 0; q < FI * 2; ++q) {
                const int fl = q * 16 + (lane >> 2), tl = (lane & 3) * 8;
                const int64_t row = f0 + wf * FI * 32 + fl;
                if (row >= g.rows_w) continue;
                float v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) v[u] = reg[(tl + u) * S::OUT_LD + fl];
                if constexpr (SYM) {
                    *reinterpret_cast<u32x4 *>((EPI == GRAM ? g.o : g.bo) + z * g.ob + row * g.ldo + tj + tl) = pack_h8(v);
                } else if constexpr (EPI == APPLY) {
                    *reinterpret_cast<u32x4 *>(g.xt + z * g.tb + row * g.ldt + tj + tl) = pack_h8(v);
                } else if (row < g.cols) {
                    uint16_t *o = static_cast<uint16_t *>(g.out) + z * g.outb + row * g.ldout + tj + tl;
                    if (tj + tl + 8 <= g.r) {
                        *reinterpret_cast<any16 *>(o) = Elt<true>::pack(v);
                    } else {
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            if (tj + tl + u < g.r) Elt<true>::store_one(o, u, v[u]);
                    }
                }
            }
        }
        __builtin_amdgcn_wave_barrier();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// The partial sums of A's K splits, added in their order, 64 x 64 values on or below the diagonal a
// workgroup, stored as they are and transposed.
__global__ __launch_bounds__(256) void gram_fold_kernel(Args g) {
    __shared__ float tile[64][65];
    const int z = blockIdx.y, mn = blockIdx.x, th = threadIdx.x;
    int ti = static_cast<int>((sqrtf(8.0f * static_cast<float>(mn) + 1.0f) - 1.0f) * 0.5f);
    while (ti * (ti + 1) / 2 > mn) --ti;
    while ((ti + 1) * (ti + 2) / 2 <= mn) ++ti;
    const int fi = mn - ti * (ti + 1) / 2;
    const int64_t one = static_cast<int64_t>(g.rows_x) * g.rows_x;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int tl = i * 32 + (th >> 3), fl = (th & 7) * 8, t = ti * 64 + tl, f = fi * 64 + fl;
        const float *p = g.part + static_cast<int64_t>(z) * g.splits * one + static_cast<int64_t>(t) * g.rows_x + f;
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int k = 0; k < g.splits; ++k) {
            const float4 x = reinterpret_cast<const float4 *>(p + k * one)[0], y = reinterpret_cast<const float4 *>(p + k * one)[1];
            v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
            v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
        }
        symmetric_values<GRAM>(g, z, t, f, v);
        *reinterpret_cast<u32x4 *>(g.o + z * g.ob + static_cast<int64_t>(t) * g.ldo + f) = pack_h8(v);
#pragma unroll
        for (int u = 0; u < 8; ++u) tile[tl][fl + u] = v[u];
    }
    if (ti == fi) return;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int fl = i * 32 + (th >> 3), tl = (th & 7) * 8;
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = tile[tl + u][fl];
        *reinterpret_cast<u32x4 *>(g.o + z * g.ob + static_cast<int64_t>(fi * 64 + fl) * g.ldo + ti * 64 + tl) = pack_h8(v);
    }
}

// ---- plan and launches ---------------------------------------------------------------------------

using Big = linear::Shape<256, 256, 2, 4, 3, 2>;    // one workgroup of eight waves per CU
using Mid = linear::Shape<128, 128, 2, 2, 2, 2>;    // two of four
using Small = linear::Shape<64, 64, 2, 2, 4, 4>;    // two of four
enum { BIG, MID, SMALL, SHAPES };
constexpr int kSide[SHAPES] = {256, 128, 64}, kThreads[SHAPES] = {512, 256, 256}, kPerCu[SHAPES] = {1, 2, 2};
static_assert(Big::BF == 256 && Mid::BF == 128 && Small::BF == 64, "sides");
// us of a step of K with as many workgroups per CU as fit, of a tile's start and end
constexpr double kStepUs[SHAPES] = {1.25, 0.70, 0.30}, kTileUs[SHAPES] = {9.0, 6.0, 4.0};
constexpr int kCus = 256, kMaxSplits = 16;

struct Plan {
    int shape, splits;
    int64_t tiles;   // of one matrix, one split
};
int64_t tiles_of(int64_t rows_x, int64_t rows_w, int side, bool sym) {
    const int64_t t = ceil_div(rows_x, side);
    return sym ? t * (t + 1) / 2 : t * ceil_div(rows_w, side);
}
Plan plan_of(int64_t batch, int64_t rows_x, int64_t rows_w, int64_t steps, bool sym, bool split) {
    Plan best{SMALL, 1, 0};
    double best_us = 1e30;
    for (int i = 0; i < SHAPES; ++i) {
        const int64_t tiles = tiles_of(rows_x, rows_w, kSide[i], sym);
        for (int sp = 1; sp <= (split ? kMaxSplits : 1) && (sp == 1 || steps / sp >= 4); ++sp) {
            const int64_t groups = batch * tiles * sp, slots = static_cast<int64_t>(kCus) * kPerCu[i];
            double us = static_cast<double>(ceil_div(groups, slots)) * (static_cast<double>(ceil_div(steps, sp)) * kStepUs[i] + kTileUs[i]);
            if (sp > 1) us += 4.0 + static_cast<double>(batch) * sp * rows_x * rows_x * 4 / 3e6;
            if (us < best_us - 1e-9) {
                best_us = us;
                best = {i, sp, tiles};
            }
        }
    }
    return best;
}

struct Layout {
    int64_t r, c, rp, cp, ldx, ldr;   // ldx: of X; ldr: of X^T, O, B
    Plan gram, poly, apply;
    size_t off_hi, off_lo, off_t0, off_t1, off_o, off_b, off_d, off_e, off_norm, off_part, bytes;
};
// Rows that lie a multiple of 4 KB apart meet in few of the caches' sets (8% of a product): 128 bytes more.
int64_t apart(int64_t padded) { return padded * 2 % 4096 == 0 ? padded + kUnit : padded; }
Layout layout(int64_t batch, int64_t rows, int64_t cols) {
    Layout L;
    L.r = std::min(rows, cols);
    L.c = std::max(rows, cols);
    L.rp = round_up(L.r, kUnit);
    L.cp = round_up(L.c, kUnit);
    L.ldx = apart(L.cp);
    L.ldr = apart(L.rp);
    L.gram = plan_of(batch, L.rp, L.rp, L.cp / kUnit, true, true);
    L.poly = plan_of(batch, L.rp, L.rp, L.rp / kUnit, true, false);
    L.apply = plan_of(batch, L.rp, L.cp, L.rp / kUnit, false, false);
    const size_t x = align256(static_cast<size_t>(batch) * L.rp * L.ldx * 2), t = align256(static_cast<size_t>(batch) * L.cp * L.ldr * 2);
    const size_t s = align256(static_cast<size_t>(batch) * L.rp * L.ldr * 2), v = align256(static_cast<size_t>(batch) * L.rp * 4);
    size_t o = 0;
    L.off_hi = o;    o += x;
    L.off_lo = o;    o += x;
    L.off_t0 = o;    o += t;
    L.off_t1 = o;    o += t;
    L.off_o = o;     o += s;
    L.off_b = o;     o += s;
    L.off_d = o;     o += v;
    L.off_e = o;     o += v;
    L.off_norm = o;  o += align256(static_cast<size_t>(batch) * kNormGroups * 8);
    L.off_part = o;
    if (L.gram.splits > 1) o += align256(static_cast<size_t>(batch) * L.gram.splits * L.rp * L.rp * 4);
    L.bytes = o;
    return L;
}

template <int EPI>
hipError_t launch_product(Args g, const Plan &p, int64_t batch, hipStream_t st) {
    g.splits = p.splits;
    g.per_batch = static_cast<int>(p.tiles * p.splits);
    g.total = static_cast<int>(batch * p.tiles * p.splits);
    g.tiles_f = static_cast<int>(ceil_div(g.rows_w, kSide[p.shape]));
    g.per_xcd = static_cast<int>(ceil_div(g.total, 8));
    const dim3 grid(static_cast<unsigned>(g.per_xcd) * 8u), block(kThreads[p.shape]);
    switch (p.shape) {
        case BIG: hipLaunchKernelGGL((ortho_kernel<Big, EPI>), grid, block, 0, st, g); break;
        case MID: hipLaunchKernelGGL((ortho_kernel<Mid, EPI>), grid, block, 0, st, g); break;
        default: hipLaunchKernelGGL((ortho_kernel<Small, EPI>), grid, block, 0, st, g); break;
    }
    return hipGetLastError();
}

}  // namespace

size_t orthogonalise_workspace_bytes(int64_t batch, int64_t rows, int64_t cols) {
    return batch > 0 ? layout(batch, rows, cols).bytes : 0;
}

hipError_t launch_orthogonalise(const OrthoArgs &a, hipStream_t st) {
    if (a.batch <= 0) return hipSuccess;
    const Layout L = layout(a.batch, a.rows, a.cols);
    char *ws = static_cast<char *>(a.workspace);
    auto half = [&](size_t off) { return reinterpret_cast<uint16_t *>(ws + off); };
    const int tall = a.rows > a.cols;
    const float s = ldexpf(1.0f, static_cast<int>(lrint(0.5 * log2(static_cast<double>(L.c)))));

    LoadArgs l{};
    l.g = a.g;
    l.ldg = a.ldg;
    l.gb = a.batch_stride;
    l.rows = a.rows;
    l.cols = a.cols;
    l.part = reinterpret_cast<double *>(ws + L.off_norm);
    l.hi = half(L.off_hi);
    l.lo = half(L.off_lo);
    l.xt = half(L.off_t0);
    l.ldx = L.ldx;
    l.ldt = L.ldr;
    l.xb = L.rp * L.ldx;
    l.tb = L.cp * L.ldr;
    l.rp = static_cast<int>(L.rp);
    l.cp = static_cast<int>(L.cp);
    l.tall = tall;
    l.s = s;
    l.eps = a.eps;
    const dim3 norm_grid(kNormGroups, static_cast<unsigned>(a.batch));
    const dim3 load_grid(static_cast<unsigned>(L.cp / 64), static_cast<unsigned>(L.rp / 64), static_cast<unsigned>(a.batch));
    hipError_t e;
    if (a.g_bf16) hipLaunchKernelGGL((norm_kernel<true>), norm_grid, dim3(256), 0, st, l);
    else hipLaunchKernelGGL((norm_kernel<false>), norm_grid, dim3(256), 0, st, l);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (a.g_bf16) hipLaunchKernelGGL((load_kernel<true>), load_grid, dim3(256), 0, st, l);
    else hipLaunchKernelGGL((load_kernel<false>), load_grid, dim3(256), 0, st, l);
    if ((e = hipGetLastError()) != hipSuccess) return e;

    Args g{};
    g.rows_x = static_cast<int>(L.rp);
    g.part = reinterpret_cast<float *>(ws + L.off_part);
    g.o = half(L.off_o);
    g.bo = half(L.off_b);
    g.ldo = L.ldr;
    g.ob = L.rp * L.ldr;
    g.d = reinterpret_cast<float *>(ws + L.off_d);
    g.e = reinterpret_cast<float *>(ws + L.off_e);
    g.a = a.a;
    g.b = a.b;
    g.c = a.c;
    g.hi = l.hi;
    g.lo = l.lo;
    g.ldh = L.ldx;
    g.hb = l.xb;
    g.ldt = L.ldr;
    g.tb = l.tb;
    g.out = a.out;
    g.ldout = a.ldo;
    g.outb = a.out_batch_stride;
    g.r = L.r;
    g.cols = L.c;
    g.tall = tall;
    for (int k = 0; k < a.steps; ++k) {
        g.w = g.x = l.hi;
        g.ldw = g.ldx = L.ldx;
        g.wb = g.xb = l.xb;
        g.rows_w = static_cast<int>(L.rp);
        g.steps = static_cast<int>(L.cp / kUnit);
        g.inv = 1.0f / (s * s);
        if ((e = launch_product<GRAM>(g, L.gram, a.batch, st)) != hipSuccess) return e;
        if (L.gram.splits > 1) {
            g.splits = L.gram.splits;
            const int64_t blocks = L.rp / 64;
            hipLaunchKernelGGL(gram_fold_kernel, dim3(static_cast<unsigned>(blocks * (blocks + 1) / 2), static_cast<unsigned>(a.batch)),
                               dim3(256), 0, st, g);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        g.w = g.x = g.o;
        g.ldw = g.ldx = L.ldr;
        g.wb = g.xb = g.ob;
        g.steps = static_cast<int>(L.rp / kUnit);
        g.inv = 1.0f / (kScaleO * kScaleO);
        if ((e = launch_product<POLY>(g, L.poly, a.batch, st)) != hipSuccess) return e;
        g.x = g.bo;
        g.w = half(k & 1 ? L.off_t1 : L.off_t0);
        g.xt = half(k & 1 ? L.off_t0 : L.off_t1);
        g.wb = l.tb;
        g.rows_w = static_cast<int>(L.cp);
        g.inv = 1.0f / s;
        e = k + 1 < a.steps ? launch_product<APPLY>(g, L.apply, a.batch, st) : launch_product<LAST>(g, L.apply, a.batch, st);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace lce
