// Matrix product of e4m3 operands with a scale for each block of 128:
//   z[t, f] = sum_b sx[t, b] sw[f / 128, b] sum_{k in b} x[t, k] w[f, k] + bias[f]
//   out     = act(z) + residual
// One matrix instruction (16 x 16 x 128) takes a whole block of K for 16 x 16 outputs.  Scales that are
// powers of two (e8m0 on both sides) are operands of that instruction, which then adds to the
// accumulators by itself; other scales take the block's product from zero and one fused multiply-add per
// value, half as many issue cycles as the matrix instruction has.
//
// Tiles, steps in flight and the swizzle are those of linear_mfma.h: a step of K is 128 bytes a row,
// one block.  The features are the rows of the instruction (its A operand), so all the features of a wave
// lie in one block of 128 rows of w and share its scale, and a lane's accumulators belong to one token a
// tile: the factor is one product per lane, tile column and step.
//
// Operand layout: lane l supplies row l % 16 of A (column of B) and, of the step's eight 16-byte chunks,
// l / 16 and 4 + l / 16; which k a byte stands for is the same in both.  Result register r of lane l is
// row 4 (l / 16) + r, column l % 16.
//
// 4096 x 8192 x 8192 takes 205 to 215 us with e8m0 scales (2.6 PFLOP/s) and 238 to 256 with fp32 ones (2.2), and
// the library's fp8 product with one scale for everything 171.  Many tokens: with e8m0 scales the matrix units
// are busy 63% of the time at the 1.94 GHz that their power leaves; with fp32 ones 51%, the rest of it the
// fused multiply-adds and what feeds them.  The steps from 420 us: barriers without a wait for all loads and LDS reads held between
// the products that they feed (276), requests spread over a step (250).  Few tokens: reading the weight, 8 x
// 6656 x 202048 252 to 262 us, 5.1 to 5.3 TB/s.  Without gain: workgroups that stay and go on to the next
// tile (250 -> 266 us: more registers, and the tile's end overlaps nothing all the same), fp32 scales of four
// blocks in one load (251 -> 253), rows a few lines apart.
#pragma once

#include "blocks_internal.h"
#include "linear_mfma.h"

namespace lce {
namespace blocks {

using dev::Elt;
using dev::u32x4;
using linear::Cols;
using linear::Epi;
using linear::f4v;
using linear::i32x4;
using linear::i32x8;
using linear::kChunks;
using linear::kLoadRows;
using linear::kOutside;
using linear::kStep;
using linear::lds_ptr;
using linear::swz;
using linear::uniform_rsrc;
static_assert(kStep == kBlock, "a step of K is a block");

struct Args {
    const unsigned char *w, *x;
    int64_t ldw, ldx;     // bytes
    int K;                // bytes of a row
    int n, M;
    int tiles_f, tiles_t, splits;
    int per_xcd;          // ceil(tiles * splits / 8)
    Scales sx, sw;
    float *part;          // splits > 1: partials [splits][n][ldpart]
    int64_t ldpart;
    Epi e;
};

// a scale as stored, for the kernel's arithmetic: an exponent byte or fp32 bits
template <bool POW2>
__device__ __forceinline__ int load_scale(const Scales &s, int64_t at) {
    if constexpr (POW2) return static_cast<const unsigned char *>(s.p)[at];
    if (s.e8m0) {   // beside an fp32 one: 255 is NaN, 0 is 2^-127
        const uint32_t e = static_cast<const unsigned char *>(s.p)[at];
        return static_cast<int>(e == 255u ? 0x7fc00000u : e == 0u ? 0x00400000u : e << 23);
    }
    return static_cast<const int *>(s.p)[at];
}

// the block's product, added to acc where the scales are powers of two
template <bool POW2>
__device__ __forceinline__ f4v block_product(i32x8 a, i32x8 b, f4v acc, int sa, int sb) {
    if constexpr (POW2) return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 0, 0, 0, sa, 0, sb);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, (f4v){0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0x7f7f7f7f, 0, 0x7f7f7f7f);
}
// Holds a value to its place in the order of the code: what forms it comes before, and volatile
// statements, LDS reads among them, stay on their sides.  (The matrix instructions have no place of their
// own, and the compiler puts every LDS read of a step ahead of the first of them.)
__device__ __forceinline__ void pin(f4v &v) { asm volatile("" : "+v"(v)::"memory"); }
__device__ __forceinline__ f4v scaled_sum(f4v t, float s, f4v acc) {
    return (f4v){fmaf(t.x, s, acc.x), fmaf(t.y, s, acc.y), fmaf(t.z, s, acc.z), fmaf(t.w, s, acc.w)};
}

// Where K is no whole number of blocks, the last step reads on into the next row, and those bytes are made
// zeros in LDS (a check of every load instead took registers that the large tile does not have).
template <class S, bool POW2>
__global__ __launch_bounds__(64 * S::NW, S::NW * S::PER_CU / 4) void blocks_kernel(Args g) {
    constexpr int FI = 2 * S::FI, TJ = 2 * S::TJ, LA = S::LA, LB = S::LB, SA = S::SA, SB = S::SB;   // 16 x 16 tiles
    __shared__ __attribute__((aligned(1024))) unsigned char lds[S::LDS];

    // the tile order of linear_kernel
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
    const int steps_total = (g.K + kStep - 1) / kStep;
    const int kbeg = static_cast<int>(static_cast<int64_t>(steps_total) * ks / g.splits);
    const int kend = static_cast<int>(static_cast<int64_t>(steps_total) * (ks + 1) / g.splits);
    const int nsteps = kend - kbeg;

    const int lane = threadIdx.x & 63, quad = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wf = wave / S::WT, wt = wave % S::WT;
    // the descriptors end with the tile's last valid row, so rows past M or n read as zeros; whole
    // 16-byte chunks that hold a value of the row are read
    const int kread = (g.K + 15) & ~15;
    const int fr = min(S::BF, g.M - f0), tr = min(S::BT, g.n - t0);
    const __amdgpu_buffer_rsrc_t rsA = uniform_rsrc(
        g.w + static_cast<int64_t>(f0) * g.ldw, static_cast<uint32_t>((fr - 1) * g.ldw + kread));
    const __amdgpu_buffer_rsrc_t rsB = uniform_rsrc(
        g.x + static_cast<int64_t>(t0) * g.ldx, static_cast<uint32_t>((tr - 1) * g.ldx + kread));

    constexpr int kMaxLoads = 8;
    static_assert(LA <= kMaxLoads && LB <= kMaxLoads, "load slots");
    uint32_t voffA[kMaxLoads], voffB[kMaxLoads];
    const int lrow = lane / kChunks, lpos = lane % kChunks;
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
    auto load_a = [&](int step, int slot_a, int j) {
        unsigned char *dst = lds + slot_a * S::A_BYTES + (j * S::NW + wave) * 1024;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsA, (lds_ptr)dst, 16, voffA[j], step * kStep, 0, 0);
    };
    auto load_b = [&](int step, int slot_b, int j) {
        unsigned char *dst = lds + SA * S::A_BYTES + slot_b * S::B_BYTES + (j * S::NW + wave) * 1024;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsB, (lds_ptr)dst, 16, voffB[j], step * kStep, 0, 0);
    };
    // 16-row tile q of an operand's tile: the lane's two chunks
    auto frag = [&](const unsigned char *tile_at, int q) {
        const int r = q * 16 + l16;
        const unsigned char *row = tile_at + r * kStep;
        const i32x4 a = *reinterpret_cast<const i32x4 *>(row + (quad ^ swz(r)) * 16);
        const i32x4 b = *reinterpret_cast<const i32x4 *>(row + ((4 + quad) ^ swz(r)) * 16);
        return (i32x8){a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    };
    // the bytes past K of the last step's tiles, which are whole in LDS: zeros
    const bool cut = g.K % kStep != 0 && kend == steps_total;
    auto clear_tail = [&](int slot_a, int slot_b) {
        const int from = g.K % kStep;
        for (int r = threadIdx.x; r < S::BF + S::BT; r += 64 * S::NW) {
            const int sw = swz(r < S::BF ? r : r - S::BF);
            unsigned char *row = r < S::BF ? lds + slot_a * S::A_BYTES + r * kStep
                                           : lds + SA * S::A_BYTES + slot_b * S::B_BYTES + (r - S::BF) * kStep;
            for (int i = from; i & 15; ++i) row[((i >> 4) ^ sw) * 16 + (i & 15)] = 0;
            for (int c = (from + 15) >> 4; c < kChunks; ++c)
                *reinterpret_cast<u32x4 *>(row + (c ^ sw) * 16) = (u32x4){0u, 0u, 0u, 0u};
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        asm volatile("s_barrier" ::: "memory");
    };
    // the wave's scales: one per token in the lanes, one of its features
    const bool has_token = lane < TJ * 16 && t0 + wt * TJ * 16 + lane < g.n;
    const int64_t sx_at = has_token ? (t0 + wt * TJ * 16 + lane) * g.sx.s_row : 0;
    const int64_t sw_at = (f0 + min(wf * FI * 16, fr - 1)) / static_cast<int>(kBlock) * g.sw.s_row;
    struct StepScales {
        int x, w;
    };
    auto load_scales = [&](int step) {
        StepScales s;
        s.x = load_scale<POW2>(g.sx, sx_at + step * g.sx.s_col);
        s.w = load_scale<POW2>(g.sw, sw_at + step * g.sw.s_col);
        return s;
    };

    f4v acc[FI][TJ];
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = (f4v){0.0f, 0.0f, 0.0f, 0.0f};

    // Requests go out in the order scales of step s + 1, w of step s + SA - 1, x of step s + SB, in step s,
    // a few with each group of products (all at once they hold up the products behind them); past the
    // last step they ask for the last one again, so that the counts stay what they are.  x of step s + SB
    // takes the place of step s's, whose fragments every wave has in registers by a barrier ahead of the
    // first of those requests: so both operands are asked for two steps ahead with five tiles of LDS.
    static_assert(SA == SB + 1, "both operands' requests of a step are for the same wait");
    constexpr int PER = (LA + LB + FI - 1) / FI, FIRST_X = LA / PER > 0 ? LA / PER : 1;
    // when step s ends, what it and the SB - 2 before it asked for may be outstanding while step s + 1 is whole
    constexpr int BEFORE = (FI - 1) * PER < LA + LB ? (FI - 1) * PER : LA + LB;
    constexpr int LEFT = (SB - 2) * (LA + LB) + BEFORE;
    static_assert(FIRST_X * PER <= LA, "x is asked for behind the barrier");
    static_assert(LEFT < 64, "vmcnt");
    const int last = nsteps - 1;
    StepScales next{};
    i32x8 b[TJ], a[2];
    f4v t[4];   // products on their way to the accumulators
    constexpr int LAG = 3;
    int f[TJ], w_scale = 0;
    auto request = [&](int s, int slot_a, int slot_b, int q) {   // request q of step s
        if (q < LA) load_a(kbeg + min(s + SA - 1, last), slot_a, q);
        else if (q < LA + LB) load_b(kbeg + min(s + SB, last), slot_b, q - LA);
    };
    auto hand_over = [&](int s, int slot_a, int slot_b) {   // step s is whole in LDS, for every wave
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LEFT) : "memory");
        asm volatile("s_barrier" ::: "memory");
        if (cut && s == last) clear_tail(slot_a, slot_b);
    };
    int sa = 0, sb = 0;   // slots of step s
    if (nsteps > 0) {
        next = load_scales(kbeg);
#pragma unroll
        for (int s = 0; s < SB; ++s)   // as steps before 0 would have asked
#pragma unroll
            for (int q = 0; q < LA + LB; ++q) request(s - SB, s, s, q);
        hand_over(0, 0, 0);
#pragma unroll
        for (int j = 0; j < TJ; ++j) b[j] = frag(lds + SA * S::A_BYTES, wt * TJ + j);
        a[0] = frag(lds, wf * FI);
        if constexpr (!POW2) {
#pragma unroll
            for (int q = 0; q < 4; ++q) t[q] = (f4v){0.0f, 0.0f, 0.0f, 0.0f};
        }
    }
    for (int s = 0; s < nsteps; ++s) {
        const int na = sa + 1 == SA ? 0 : sa + 1, nb = sb + 1 == SB ? 0 : sb + 1;
        const unsigned char *At = lds + sa * S::A_BYTES;
        const unsigned char *An = lds + na * S::A_BYTES, *Bn = lds + SA * S::A_BYTES + nb * S::B_BYTES;
        // a lane's token of tile j is lane 16 j + l % 16 of the wave's
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            f[j] = __builtin_amdgcn_ds_bpermute((j * 16 + l16) * 4, next.x);
            if constexpr (!POW2) f[j] = __float_as_int(__int_as_float(f[j]) * __int_as_float(next.w));
        }
        w_scale = next.w;
        next = load_scales(kbeg + min(s + 1, last));
        const int fa = sa == 0 ? SA - 1 : sa - 1;   // free since the last step ended
#pragma unroll
        for (int i = 0; i < FI; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            if (i == FIRST_X) {
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // b, which the first products have used
                asm volatile("s_barrier" ::: "memory");
            }
            if (i + 1 < FI) {
#pragma unroll
                for (int q = i * PER; q < (i + 1) * PER; ++q) request(s, fa, sb, q);
            }
            if (i + 1 < FI) {
                a[(i + 1) & 1] = frag(At, wf * FI + i + 1);
            } else {   // the wave has read all of step s; the next one's operands follow the last products
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                hand_over(s + 1, na, nb);
                a[0] = frag(An, wf * FI);
#pragma unroll
                for (int q = i * PER; q < LA + LB; ++q) request(s, fa, sb, q);
            }
#pragma unroll
            for (int j = 0; j < TJ; ++j) {
                const int q = i * TJ + j;
                if constexpr (POW2) {
                    acc[i][j] = block_product<true>(a[i & 1], b[j], acc[i][j], w_scale, f[j]);
                } else {   // a product is added LAG later, when it has left the matrix core
                    t[q & 3] = block_product<false>(a[i & 1], b[j], t[q & 3], 0, 0);
                    pin(t[q & 3]);
                    if (q >= LAG) {
                        const int pi = (q - LAG) / TJ, pj = (q - LAG) % TJ;
                        acc[pi][pj] = scaled_sum(t[(q - LAG) & 3], __int_as_float(f[pj]), acc[pi][pj]);
                        pin(acc[pi][pj]);
                    }
                }
                if (i + 1 == FI) {
                    if constexpr (POW2) pin(acc[i][j]);
                    b[j] = frag(Bn, wt * TJ + j);
                }
            }
            if constexpr (POW2) {
#pragma unroll
                for (int j = 0; j < TJ; ++j) pin(acc[i][j]);
            }
        }
        if constexpr (!POW2) {
#pragma unroll
            for (int q = FI * TJ - LAG; q < FI * TJ; ++q)
                acc[q / TJ][q % TJ] = scaled_sum(t[q & 3], __int_as_float(f[q % TJ]), acc[q / TJ][q % TJ]);
        }
        sa = na;
        sb = nb;
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __syncthreads();   // every wave is done with the operand tiles, and nothing is on its way there

    // epilogue: a wave's own LDS region, 32 tokens at a time
    constexpr int LPT = FI * 2, TPP = 64 / LPT;   // lanes per token, tokens per pass
    constexpr int PASSES = 32 / TPP, U = PASSES < 4 ? PASSES : 4;
    float *reg = reinterpret_cast<float *>(lds) + wave * 32 * S::OUT_LD;
    const int lf = (lane % LPT) * 8;
    const int64_t fcol = f0 + wf * FI * 16 + lf;
    const bool split = g.splits > 1;
    Cols cols;
    if (!split) cols = linear::load_cols(g.e, fcol);
#pragma unroll
    for (int jj = 0; jj < TJ; jj += 2) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < FI; ++i)
                *reinterpret_cast<f4v *>(reg + (j * 16 + l16) * S::OUT_LD + i * 16 + quad * 4) = acc[i][jj + j];
        __builtin_amdgcn_wave_barrier();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll 1
        for (int p0 = 0; p0 < PASSES; p0 += U) {
            const int tl = p0 * TPP + lane / LPT;
            const int64_t t = t0 + (wt * TJ + jj) * 16 + tl;
            auto read = [&](float (&v)[U][8]) {
#pragma unroll
                for (int p = 0; p < U; ++p) {
                    const float4 x = *reinterpret_cast<const float4 *>(reg + (tl + p * TPP) * S::OUT_LD + lf);
                    const float4 y = *reinterpret_cast<const float4 *>(reg + (tl + p * TPP) * S::OUT_LD + lf + 4);
                    v[p][0] = x.x; v[p][1] = x.y; v[p][2] = x.z; v[p][3] = x.w;
                    v[p][4] = y.x; v[p][5] = y.y; v[p][6] = y.z; v[p][7] = y.w;
                }
            };
            if (fcol >= g.M) continue;
            if (!split) {
                linear::finish<U>(g.e, cols, t, TPP, fcol, read);
            } else {   // ldpart is M in whole eights
                float v[U][8];
                read(v);
#pragma unroll
                for (int p = 0; p < U; ++p) {
                    if (t + p * TPP >= g.n) continue;
                    float4 *o = reinterpret_cast<float4 *>(
                        g.part + (static_cast<int64_t>(ks) * g.n + t + p * TPP) * g.ldpart + fcol);
                    o[0] = make_float4(v[p][0], v[p][1], v[p][2], v[p][3]);
                    o[1] = make_float4(v[p][4], v[p][5], v[p][6], v[p][7]);
                }
            }
        }
        __builtin_amdgcn_wave_barrier();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// The partial sums of the K splits, added in their order, through the epilogue.  All loads of up to SPLITS of
// them are under way at once; the last one's again where there are fewer.
template <int SPLITS>
__global__ __launch_bounds__(256) void blocks_fold_kernel(const float *part, int64_t ldpart, int splits, Epi e) {
    const int64_t per = ldpart / 8, total = e.n * per;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t t = i / per, f = (i - t * per) * 8;
        const float4 *p = reinterpret_cast<const float4 *>(part + t * ldpart + f);
        const int64_t step = e.n * ldpart / 4;
        float4 x[SPLITS], y[SPLITS];
#pragma unroll
        for (int k = 0; k < SPLITS; ++k) {
            x[k] = p[min(k, splits - 1) * step];
            y[k] = p[min(k, splits - 1) * step + 1];
        }
        const Cols c = linear::load_cols(e, f);
        linear::finish<1>(e, c, t, 0, f, [&](float (&s)[1][8]) {
            float v[8] = {x[0].x, x[0].y, x[0].z, x[0].w, y[0].x, y[0].y, y[0].z, y[0].w};
#pragma unroll
            for (int k = 1; k < SPLITS; ++k) {
                const float q[8] = {x[k].x, x[k].y, x[k].z, x[k].w, y[k].x, y[k].y, y[k].z, y[k].w};
#pragma unroll
                for (int u = 0; u < 8; ++u) v[u] = k < splits ? v[u] + q[u] : v[u];
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) s[0][u] = v[u];
        });
    }
}

// ---- few tokens ------------------------------------------------------------------------
//
// Up to 32 tokens, as linear_rows_kernel: a workgroup takes 16 features and its eight waves an eighth of
// the blocks of K each; operands go straight from memory to registers, U blocks ahead of those in use.
// It wins while a launch's length is that of its chains (8 x 4096 x 4096 9.2 us; 64 x 32 tiles split along K
// take a second launch); where the weight's bytes bound the call it reaches 3.7 TB/s and the tiles take over
// (8 x 6656 x 202048 359 us, tiles of 64 x 32 257).
constexpr int kRowsWaves = 8;

template <bool POW2, bool CUT, int TT>   // CUT: K is no multiple of 16; TT: token tiles of 16
__global__ __launch_bounds__(64 * kRowsWaves, 2) void blocks_rows_kernel(Args g) {
    constexpr int U = TT == 1 ? 4 : 2;   // blocks at once
    __shared__ __attribute__((aligned(16))) float sums[kRowsWaves][TT * 256];
    const int lane = threadIdx.x & 63, quad = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int f0 = blockIdx.x * 16;
    const int rows = min(16, g.M - f0);
    const int kread = (g.K + 15) & ~15;
    const __amdgpu_buffer_rsrc_t rsW = uniform_rsrc(
        g.w + static_cast<int64_t>(f0) * g.ldw, static_cast<uint32_t>((rows - 1) * g.ldw + kread));
    const __amdgpu_buffer_rsrc_t rsX = uniform_rsrc(g.x, static_cast<uint32_t>((g.n - 1) * g.ldx + kread));
    const uint32_t vw = static_cast<uint32_t>(l16) * static_cast<uint32_t>(g.ldw) + quad * 16;
    uint32_t vx[TT];
    int64_t sx_at[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        vx[t] = static_cast<uint32_t>(t * 16 + l16) * static_cast<uint32_t>(g.ldx) + quad * 16;
        sx_at[t] = (t * 16 + l16 < g.n ? t * 16 + l16 : 0) * g.sx.s_row;
    }
    const int64_t sw_at = f0 / static_cast<int>(kBlock) * g.sw.s_row;
    const int total = (g.K + kStep - 1) / kStep;
    const int beg = static_cast<int>(static_cast<int64_t>(total) * wave / kRowsWaves);
    const int end = static_cast<int>(static_cast<int64_t>(total) * (wave + 1) / kRowsWaves);
    struct Set {
        u32x4 w[U][2], x[TT][U][2];
        int sx[TT][U], sw[U];
    };
    auto fetch = [&](int s, Set &q) {   // zeros past this wave's share and past K
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (s + u) * kStep, at = s + u < end ? s + u : end - 1;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool in = s + u < end && k + h * 64 + quad * 16 < g.K;
                q.w[u][h] = __builtin_amdgcn_raw_buffer_load_b128(rsW, in ? vw + k + h * 64 : kOutside, 0, 0);
#pragma unroll
                for (int t = 0; t < TT; ++t)
                    q.x[t][u][h] = __builtin_amdgcn_raw_buffer_load_b128(rsX, in ? vx[t] + k + h * 64 : kOutside, 0, 0);
            }
            q.sw[u] = load_scale<POW2>(g.sw, sw_at + at * g.sw.s_col);
#pragma unroll
            for (int t = 0; t < TT; ++t) q.sx[t][u] = load_scale<POW2>(g.sx, sx_at[t] + at * g.sx.s_col);
        }
    };
    f4v acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = (f4v){0.0f, 0.0f, 0.0f, 0.0f};
    // bytes of the chunk at k that lie past K: zeros
    auto trim = [&](u32x4 &v, int k) {
        const int keep = g.K - k;
        if (keep >= 16) return;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int left = keep - 4 * d;
            v[d] = left >= 4 ? v[d] : left <= 0 ? 0u : v[d] & ((1u << (8 * left)) - 1u);
        }
    };
    auto use = [&](int s, Set &q) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u >= end) break;   // a scale may be anything where there is no block
            auto join = [&](u32x4 (&v)[2]) {
                if constexpr (CUT) {
                    trim(v[0], (s + u) * kStep + quad * 16);
                    trim(v[1], (s + u) * kStep + 64 + quad * 16);
                }
                return (i32x8){static_cast<int>(v[0].x), static_cast<int>(v[0].y), static_cast<int>(v[0].z), static_cast<int>(v[0].w),
                               static_cast<int>(v[1].x), static_cast<int>(v[1].y), static_cast<int>(v[1].z), static_cast<int>(v[1].w)};
            };
            const i32x8 w = join(q.w[u]);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const f4v p = block_product<POW2>(w, join(q.x[t][u]), acc[t], q.sw[u], q.sx[t][u]);
                acc[t] = POW2 ? p : scaled_sum(p, __int_as_float(q.sx[t][u]) * __int_as_float(q.sw[u]), acc[t]);
            }
        }
    };
    if (beg < end) {
        Set s0, s1;
        fetch(beg, s0);
        for (int s = beg; s < end; s += 2 * U) {
            fetch(s + U, s1);
            use(s, s0);
            fetch(s + 2 * U, s0);
            use(s + U, s1);
        }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t)
        *reinterpret_cast<f4v *>(&sums[wave][t * 256 + l16 * 16 + quad * 4]) = acc[t];
    __syncthreads();
    const Epi &e = g.e;
    const int i = threadIdx.x;
    if (i >= TT * 256) return;
    const int64_t t = i >> 4, f = f0 + (i & 15);
    if (t >= e.n || f >= e.M) return;
    float v = sums[0][i];
#pragma unroll
    for (int k = 1; k < kRowsWaves; ++k) v += sums[k][i];
    if (e.bias) v += e.bias_bf16 ? Elt<true>::load_one(e.bias, f) : static_cast<const float *>(e.bias)[f];
    if (e.preact) Elt<true>::store_one(e.preact, t * e.ldp + f, v);
    v = linear::activate(e.act, v);
    if (e.residual) v += Elt<true>::load_one(e.residual, t * e.ldr + f);
    Elt<true>::store_one(e.out, t * e.ldo + f, v);
}

}  // namespace blocks
}  // namespace lce
