// Orthogonalised update by Newton-Schulz products, over X = G / (||G||_F + eps) with r rows and c >= r
// columns (G transposed if it is taller than wide), `steps` times:
//   A = X X^T,   B = b A + c A A,   X <- a X + B X
//
// The three products run on the matrix cores in fp16, whose 11 bits keep eight times what bf16 does at the
// same rate, with fp32 sums.  What would be lost is kept where it costs nothing:
//   X      fp16 and what that leaves in fp16, 22 bits together.  X X^T reads the first, a X both, and B X both
//          where that shows (ortho_plan.h).  What the steps make of a gradient of few directions hangs on it: held
//          in 15 bits and with fp16's X in B X, X picked up directions that grow by a step each (64 x 64 of one
//          direction 6.0e-3 of the result in five steps, 1.6e-1 in eight; now 6.0e-4 and 2.1e-3).
//   A, B   their diagonals in fp32 vectors, the rest in fp16.  X approaches orthogonal rows, so A
//          approaches its diagonal: A = D + O gives A A = O O + (D_t + D_f) O + D^2, and B X = diag X + rest.
// With these roundings put into the definition (gaussian matrices with even and uneven rows, of 1 to 16
// directions, and with singular values that fall as 1 / k), five default steps are off by up to 1.4e-3 of the
// result in the Frobenius norm and 1.9e-3 in the 2-norm from 64 rows on, and by up to 5e-3 and 6e-3 below; the
// bf16 output rounds at 1.7e-3.
// Powers of two keep fp16 in range, for the default coefficients X times 2^14 (its values are at most 1.21), O times
// 2^10 and B times 2^8 (ortho_plan.h).
//
// A and A A are symmetric: only tiles on and below the diagonal are computed, and stored a second time
// transposed.  All operands have K contiguous: X for A, O for O O, and for B X also X^T, which the
// product that forms X writes beside it (its rest behind it in each row, B's rows starting again there).
// A step is three launches, r^2 c + r^3 + 2 r^2 c operations, another 2 r^2 c with the rest (two launches where
// B, of 64 rows at most, is formed by the workgroups that use it).  Everything is padded with zeros to multiples
// of 64, so the products meet no edges.
//
// 4096 x 16384 in five steps takes 4.9 to 5.0 ms, 0.89 to 0.91 PFLOP/s where a library fp16 product reaches
// 1.4 to 1.5: a step is X X^T (321 to 332 us, 136 tiles on 256 compute units, whose matrix units are busy 41% of the time),
// A A (92 to 99, the same tiles and a quarter of the depth) and B X (554 to 569; busy 54% at the 1.7 GHz that
// their power leaves; 440 of it the main loop, the rest its ends, which read and write 0.7 GB of X).  Small
// ones are their launches: 256 x 1024, 17 launches, 98 us from a graph, 9 of them for the rest in B X.
// The steps: tiles chosen for each product, instructions held in place between LDS reads (1003 x 517 x 4 161 ->
// 149 us, 2048 x 2048 886 -> 380).
#include <hip/hip_runtime.h>
#include <algorithm>
#include <math.h>
#include <stdint.h>

#include "blocks_internal.h"
#include "ce_device.h"
#include "linear_mfma.h"
#include "ortho_plan.h"

namespace lce {
namespace {

using namespace ortho_plan;

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
constexpr int kNormGroups = 1024;         // partial sums of squares per matrix, at most

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

__device__ __forceinline__ u32x4 pack_h8(const float (&v)[8]) {
    h8 h;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = static_cast<_Float16>(v[e]);
    return __builtin_bit_cast(u32x4, h);
}

typedef _Float16 h4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint2 pack_h4(const float (&v)[4]) {
    return __builtin_bit_cast(uint2, (h4){static_cast<_Float16>(v[0]), static_cast<_Float16>(v[1]), static_cast<_Float16>(v[2]), static_cast<_Float16>(v[3])});
}

// Holds a matrix instruction to its place in the order of the code (blocks_mfma.h).  In the accumulation
// registers: where a wave has more than 256, the compiler keeps sums there, and copies them both ways for
// a place in the vector registers (2048 x 2048 in all: 886 us for 380).
__device__ __forceinline__ void pin(f16v &v) { asm volatile("" : "+a"(v)::"memory"); }
// What fp16 leaves of eight values, in fp16
__device__ __forceinline__ u32x4 pack_rest(const float (&v)[8]) {
    h8 h;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = static_cast<_Float16>(v[e] - static_cast<float>(static_cast<_Float16>(v[e])));
    return __builtin_bit_cast(u32x4, h);
}
__device__ __forceinline__ void unpack(u32x4 hi, u32x4 lo, float (&v)[8]) {   // exact: 22 bits
    const h8 h = __builtin_bit_cast(h8, hi), l = __builtin_bit_cast(h8, lo);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = static_cast<float>(h[e]) + static_cast<float>(l[e]);
}

// eight values of a row from column c on, zeros from `cols` on
template <bool BF16>
__device__ __forceinline__ void load8(const void *p, int64_t row, int64_t c, int64_t cols, float (&v)[8]) {
    if (c + 8 <= cols) {
        if constexpr (BF16) {
            const u32x4 q = *reinterpret_cast<const any16 *>(static_cast<const uint16_t *>(p) + row + c);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = Elt<true>::get(q, e);
        } else {
            const any16 *q = reinterpret_cast<const any16 *>(static_cast<const float *>(p) + row + c);
            const u32x4 x = q[0], y = q[1];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = Elt<false>::get(e < 4 ? x : y, e & 3);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = c + e < cols ? Elt<BF16>::load_one(p, row + c + e) : 0.0f;
    }
}

// ---- the norm, and X in fp16 -----------------------------------------------------------------

struct LoadArgs {
    const void *g;
    int64_t ldg, gb;                  // strides of G (elements)
    int64_t rows, cols;               // of G
    double *part;                     // [batch][kNormGroups], the first `groups` used
    int groups;
    uint16_t *hi, *lo, *xt;           // X and its rest [rp][ldx], X^T [cp][ldt]
    int64_t ldx, ldt, xb, tb;         // row and batch strides (elements)
    int rp, cp;                       // padded rows and columns of X
    int rest_at;                      // X^T: where in a row the rest's starts, 0: not wanted
    int tall;                         // X is G^T
    float s, eps;
};

// Sums of squares in fp64, a fixed share of the rows' 2048-value pieces per workgroup: no square of a
// finite fp32 value overflows, and the order is fixed.  (4096 x 16384 bf16: 35 us, 3.8 TB/s.)
template <bool BF16>
__global__ __launch_bounds__(256) void norm_kernel(LoadArgs a) {
    __shared__ double sums[4];
    const int64_t pieces = (a.cols + 2047) / 2048, total = a.rows * pieces;
    const int64_t base = blockIdx.y * a.gb;
    double sum = 0.0;
    for (int64_t i = blockIdx.x; i < total; i += gridDim.x) {
        const int64_t row = i / pieces, c = (i - row * pieces) * 2048 + threadIdx.x * 8;
        float v[8];
        load8<BF16>(a.g, base + row * a.ldg, c, c < a.cols ? a.cols : 0, v);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            // two squares of 24-bit values in fp64 are exact; their sum rounds once
            sum += static_cast<double>(v[e]) * static_cast<double>(v[e]) + static_cast<double>(v[e + 1]) * static_cast<double>(v[e + 1]);
        }
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) a.part[blockIdx.y * kNormGroups + blockIdx.x] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// A workgroup takes 64 x 64 of X: hi, lo and the transposed hi (and lo, where B X takes it), zeros in the padding
// (4096 x 16384 bf16: 97 us, 5.5 TB/s of what it reads and writes).
template <bool BF16>
__global__ __launch_bounds__(256) void load_kernel(LoadArgs a) {
    __shared__ float tile[64][65];
    __shared__ double sums[4];
    const int t = threadIdx.x, z = blockIdx.z;
    const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;   // of X
    const int g0 = a.tall ? c0 : r0, h0 = a.tall ? r0 : c0;   // of G
    float v[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t row = g0 + i * 32 + (t >> 3);
        load8<BF16>(a.g, z * a.gb + row * a.ldg, h0 + (t & 7) * 8, row < a.rows ? a.cols : 0, v[i]);
    }
    double s = 0.0;
    for (int i = t; i < a.groups; i += 256) s += a.part[z * kNormGroups + i];
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) s += __shfl_xor(s, m);
    if ((t & 63) == 0) sums[t >> 6] = s;
    __syncthreads();
    s = (sums[0] + sums[1]) + (sums[2] + sums[3]);
    // fp64: of the smallest and the largest fp32 values the factor is no normal fp32 number
    const double factor = static_cast<double>(a.s) / (sqrt(s) + static_cast<double>(a.eps));
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) tile[i * 32 + (t >> 3)][(t & 7) * 8 + e] = static_cast<float>(v[i][e] * factor);
    __syncthreads();
    // eight values along a row of X, and along a row of X^T
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int line = i * 32 + (t >> 3), at = (t & 7) * 8;
        float p[8], q[8];
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
        const int64_t x_at = z * a.xb + static_cast<int64_t>(r0 + line) * a.ldx + c0 + at;
        *reinterpret_cast<u32x4 *>(a.hi + x_at) = pack_h8(p);
        *reinterpret_cast<u32x4 *>(a.lo + x_at) = pack_rest(p);
        uint16_t *xt = a.xt + z * a.tb + static_cast<int64_t>(c0 + line) * a.ldt + r0 + at;
        *reinterpret_cast<u32x4 *>(xt) = pack_h8(q);
        if (a.rest_at) *reinterpret_cast<u32x4 *>(xt + a.rest_at) = pack_rest(q);
    }
}

// ---- products ----------------------------------------------------------------------------------

enum { GRAM, POLY, APPLY, LAST };

struct Args {
    const uint16_t *w, *x;            // K contiguous: features [rows_w][ldw], tokens [rows_x][ldx]
    int64_t ldw, ldx, wb, xb;         // row and batch strides (elements)
    int rows_w, rows_x;               // multiples of 64
    int steps, steps_x;               // of K; of x's, which starts again at its end (APPLY, LAST)
    int tiles_f, per_batch, total;    // tiles: per row of them, of one matrix, of all
    int groups, per_xcd;              // workgroups; ceil(groups / 8)
    float *part;                      // groups != total: [2 groups][side][side] fp32
    // epilogue
    float inv, inv_poly;              // of the products' scale; apply_short_kernel: of O O's
    float so, sb, inv_o, inv_b;       // what O and B are held times, and their inverses
    uint16_t *o;                      // O [rows][ldo]: written by GRAM, read by POLY
    uint16_t *bo;                     // B's off-diagonal part
    int64_t ldo, ob;
    float *d, *e;                     // diagonals of A, and a + that of B: [batch][rows]
    float a, b, c;
    uint16_t *hi, *lo, *xt;           // X, its rest and the next X^T
    int rest_at;                      // of X^T
    int64_t ldh, hb, ldt, tb;
    void *out;                        // LAST: bf16
    int64_t ldout, outb;
    int64_t r, cols;                  // of X, not padded
    int tall;
};

// Tile mn of a lower triangle, row ti of which holds ti + 1
__device__ __forceinline__ void triangle(int mn, int &ti, int &fi) {
    ti = static_cast<int>((sqrtf(8.0f * static_cast<float>(mn) + 1.0f) - 1.0f) * 0.5f);
    while (ti * (ti + 1) / 2 > mn) --ti;
    while ((ti + 1) * (ti + 2) / 2 <= mn) ++ti;
    fi = mn - ti * (ti + 1) / 2;
}

// Values v of A, N of row t from column f on, to O and its diagonal
template <int N>
__device__ __forceinline__ void gram_values(const Args &g, int z, int t, int f, float (&v)[N]) {
#pragma unroll
    for (int u = 0; u < N; ++u) {
        v[u] *= g.inv;
        if (t == f + u) {
            g.d[static_cast<int64_t>(z) * g.rows_x + t] = v[u];
            v[u] = 0.0f;
        }
        v[u] *= g.so;
    }
}
// The same, or (POLY) values of O O to B, from O there, the diagonal at t and at f .. f + 7
template <int EPI>
__device__ __forceinline__ void symmetric_values(const Args &g, int z, int t, int f, u32x4 oq, float dt, const float (&df)[8], float (&v)[8]) {
    if constexpr (EPI == GRAM) {
        gram_values(g, z, t, f, v);
    } else {
        const h8 o = __builtin_bit_cast(h8, oq);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const float ov = static_cast<float>(o[u]) * g.inv_o;
            float square = fmaf(dt + df[u], ov, v[u] * g.inv);
            if (t == f + u) {
                square = fmaf(dt, dt, square);   // O is 0 there
                g.e[static_cast<int64_t>(z) * g.rows_x + t] = g.a + fmaf(g.c, square, g.b * dt);
                v[u] = 0.0f;
            } else {
                v[u] = fmaf(g.c, square, g.b * ov) * g.sb;
            }
        }
    }
}

// APPLY and LAST: the product's values v of eight features of a token to X' in all its forms, but for the
// transposed one.  LAST leaves what the output's transpose holds in v.
template <int EPI>
__device__ __forceinline__ void apply_values(const Args &g, int z, int t, int f, u32x4 hi, u32x4 lo, float et, float (&v)[8]) {
    float was[8];
    unpack(hi, lo, was);
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = fmaf(et, was[u], v[u] * g.inv_b);
    if constexpr (EPI == APPLY) {
        const int64_t at = z * g.hb + static_cast<int64_t>(t) * g.ldh + f;
        *reinterpret_cast<u32x4 *>(g.hi + at) = pack_h8(v);
        *reinterpret_cast<u32x4 *>(g.lo + at) = pack_rest(v);
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
// Eight tokens of one feature: the mirrored tile, X^T, or a row of a tall output
template <int EPI>
__device__ __forceinline__ void turned_values(const Args &g, int z, int64_t row, int t, const float (&v)[8]) {
    if constexpr (EPI == GRAM || EPI == POLY) {
        *reinterpret_cast<u32x4 *>((EPI == GRAM ? g.o : g.bo) + z * g.ob + row * g.ldo + t) = pack_h8(v);
    } else if constexpr (EPI == APPLY) {
        uint16_t *o = g.xt + z * g.tb + row * g.ldt + t;
        *reinterpret_cast<u32x4 *>(o) = pack_h8(v);
        if (g.rest_at) *reinterpret_cast<u32x4 *>(o + g.rest_at) = pack_rest(v);
    } else if (row < g.cols) {
        uint16_t *o = static_cast<uint16_t *>(g.out) + z * g.outb + row * g.ldout + t;
        if (t + 8 <= g.r) {
            *reinterpret_cast<any16 *>(o) = Elt<true>::pack(v);
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (t + u < g.r) Elt<true>::store_one(o, u, v[u]);
        }
    }
}
template <int EPI>
__device__ __forceinline__ void symmetric_store(const Args &g, int z, int t, int f, const float (&v)[8]) {
    *reinterpret_cast<u32x4 *>((EPI == GRAM ? g.o : g.bo) + z * g.ob + static_cast<int64_t>(t) * g.ldo + f) = pack_h8(v);
}

// The steps of all tiles are one sequence, cut into equal ranges: the unit at which range i of n starts
__device__ __forceinline__ int64_t range_start(int64_t units, int n, int i) { return units * i / n; }

template <class S, int EPI>
__global__ __launch_bounds__(64 * S::NW, S::NW * S::PER_CU / 4) void ortho_kernel(Args g) {
    constexpr int FI = S::FI, TJ = S::TJ, KK = 4, LA = S::LA, LB = S::LB, SA = S::SA, SB = S::SB;
    constexpr bool SYM = EPI == GRAM || EPI == POLY;
    static_assert(!SYM || S::BF == S::BT, "tiles of a symmetric product are square");
    __shared__ __attribute__((aligned(1024))) unsigned char lds[S::LDS];

    // Each XCD takes a contiguous range of the workgroups' ranges.  With as many workgroups as tiles a range
    // is a tile.  Otherwise ranges start and end inside tiles, and what a workgroup has of such a tile goes
    // to memory: slot 2 w for the piece that its range starts with, 2 w + 1 for one that it ends with.
    const int w = (blockIdx.x & 7) * g.per_xcd + (blockIdx.x >> 3);
    if (static_cast<int>(blockIdx.x >> 3) >= g.per_xcd || w >= g.groups) return;
    const bool whole = EPI != GRAM || g.groups == g.total;
    int tile = w, s0 = 0, left = g.steps;   // left: steps of the range
    if (!whole) {
        const int64_t units = static_cast<int64_t>(g.total) * g.steps, from = range_start(units, g.groups, w);
        left = __builtin_amdgcn_readfirstlane(static_cast<int>(range_start(units, g.groups, w + 1) - from));
        tile = __builtin_amdgcn_readfirstlane(static_cast<int>(from / g.steps));
        s0 = __builtin_amdgcn_readfirstlane(static_cast<int>(from - static_cast<int64_t>(tile) * g.steps));
    }

    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wf = wave / S::WT, wt = wave % S::WT;
    const uint32_t ldw = static_cast<uint32_t>(g.ldw * 2), ldx = static_cast<uint32_t>(g.ldx * 2);
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
    while (left > 0) {
    const int z = __builtin_amdgcn_readfirstlane(tile / g.per_batch), mn = tile - z * g.per_batch;
    int ti, fi;
    if constexpr (SYM) {
        triangle(mn, ti, fi);
    } else {   // groups of four token tiles, its token tiles fastest
        constexpr int GROUP = 4;
        const int tiles_t = g.per_batch / g.tiles_f;
        const int first_t = mn / (GROUP * g.tiles_f) * GROUP;
        const int gt = min(GROUP, tiles_t - first_t);
        const int within = mn - first_t * g.tiles_f;
        ti = first_t + within % gt;
        fi = within / gt;
    }
    const int t0 = __builtin_amdgcn_readfirstlane(ti * S::BT), f0 = __builtin_amdgcn_readfirstlane(fi * S::BF);
    const int kbeg = s0, nsteps = min(left, g.steps - s0), steps_x = SYM ? g.steps : g.steps_x;
    const int fr = min(S::BF, g.rows_w - f0), tr = min(S::BT, g.rows_x - t0);
    const __amdgpu_buffer_rsrc_t rsA = uniform_rsrc(g.w + z * g.wb + f0 * g.ldw, (fr - 1) * ldw + g.steps * kStep);
    const __amdgpu_buffer_rsrc_t rsB = uniform_rsrc(g.x + z * g.xb + t0 * g.ldx, (tr - 1) * ldx + steps_x * kStep);
    const int last = nsteps - 1;
    // request q of a step: w of step sw, then x of step sx
    auto request = [&](int sw, int sx, int slot_a, int slot_b, int q) {
        if (q < LA)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsA, (lds_ptr)(lds + slot_a * S::A_BYTES + (q * S::NW + wave) * 1024), 16,
                                                     voffA[q < LA ? q : 0], (kbeg + min(sw, last)) * kStep, 0, 0);
        else if (q < LA + LB)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsB, (lds_ptr)(lds + SA * S::A_BYTES + slot_b * S::B_BYTES + ((q - LA) * S::NW + wave) * 1024), 16,
                voffB[q < LA ? 0 : q - LA],
                (kbeg + min(sx, last) - (SYM || kbeg + min(sx, last) < steps_x ? 0 : steps_x)) * kStep, 0, 0);
    };
    auto frag = [&](const unsigned char *tile_at, int q, int kk) {   // 32-row tile q, instruction kk of the step
        const int r = q * 32 + (lane & 31);
        return *reinterpret_cast<const h8 *>(tile_at + r * kStep + ((kk * 2 + half) ^ swz(r)) * 16);
    };
    // The schedule of blocks_kernel (blocks_mfma.h): requests run ahead by as many steps as LDS holds and are
    // spread over a step; past the last step they ask for the last one again.  With two or more tiles of
    // features to a wave, x of step s + SB takes the place of step s's once every wave has that in registers.
    constexpr bool EARLY = FI >= 2;
    static_assert(SA == SB + (EARLY ? 1 : 0), "both operands' requests of a step are for the same wait");
    constexpr int AHEAD = EARLY ? SB : SB - 1;   // steps
    constexpr int PER = (LA + LB + FI - 1) / FI, FIRST_X = LA / PER > 0 ? LA / PER : 1;
    constexpr int BEFORE = (FI - 1) * PER < LA + LB ? (FI - 1) * PER : LA + LB;
    // when a step ends, what it (its first groups) and the AHEAD - 2 before it asked for may be outstanding
    // while the next is whole
    constexpr int LEFT = EARLY ? (AHEAD - 2) * (LA + LB) + BEFORE : (AHEAD - 1) * (LA + LB);
    static_assert((!EARLY || FIRST_X * PER <= LA) && LEFT < 64 && LEFT >= 0, "requests");
    f16v acc[FI][TJ];
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = (f16v){};
    h8 b[TJ][KK], a[2][KK];
#pragma unroll
    for (int s = 0; s < AHEAD; ++s)
#pragma unroll
        for (int q = 0; q < LA + LB; ++q) request(s, s, s, s, q);
    auto hand_over = [&]() {   // the next step is whole in LDS, for every wave
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LEFT) : "memory");
        asm volatile("s_barrier" ::: "memory");
    };
    if constexpr (EARLY) {   // all of the first requests but the last step's
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((AHEAD - 1) * (LA + LB)) : "memory");
        asm volatile("s_barrier" ::: "memory");
    } else {
        hand_over();
    }
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
#pragma unroll
        for (int j = 0; j < TJ; ++j) b[j][kk] = frag(lds + SA * S::A_BYTES, wt * TJ + j, kk);
        a[0][kk] = frag(lds, wf * FI, kk);
    }
    int sa = 0, sb = 0;   // slots of the present step
    for (int s = 0; s < nsteps; ++s) {
        const int na = sa + 1 == SA ? 0 : sa + 1, nb = sb + 1 == SB ? 0 : sb + 1;
        const int fa = sa == 0 ? SA - 1 : sa - 1, fb = EARLY ? sb : sb == 0 ? SB - 1 : sb - 1;   // free, or about to be
        const unsigned char *At = lds + sa * S::A_BYTES;
        const unsigned char *An = lds + na * S::A_BYTES, *Bn = lds + SA * S::A_BYTES + nb * S::B_BYTES;
#pragma unroll
        for (int i = 0; i < FI; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            if (EARLY && i == FIRST_X) {
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // b, which the first products have used
                asm volatile("s_barrier" ::: "memory");
            }
            if (i + 1 < FI) {
#pragma unroll
                for (int q = i * PER; q < (i + 1) * PER; ++q) request(s + SA - 1, s + AHEAD, fa, fb, q);
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) a[(i + 1) & 1][kk] = frag(At, wf * FI + i + 1, kk);
            } else {
                if constexpr (!EARLY) {
#pragma unroll
                    for (int q = 0; q < LA + LB; ++q) request(s + AHEAD, s + AHEAD, fa, fb, q);
                }
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                hand_over();
                if constexpr (EARLY) {
#pragma unroll
                    for (int q = i * PER; q < LA + LB; ++q) request(s + SA - 1, s + AHEAD, fa, fb, q);
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk) a[FI & 1][kk] = frag(An, wf * FI, kk);
                }
            }
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
#pragma unroll
                for (int j = 0; j < TJ; ++j) {
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[i & 1][kk], b[j][kk], acc[i][j], 0, 0, 0);
                    pin(acc[i][j]);
                    if (i + 1 == FI) b[j][kk] = frag(Bn, wt * TJ + j, kk);
                }
                if (i + 1 == FI && !EARLY) a[0][kk] = frag(An, wf * FI, kk);
            }
        }
        sa = na;
        sb = nb;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

    // epilogue: a wave's own LDS region, 32 tokens at a time, eight features of a token per lane; what it
    // reads of X or O for them is asked for all at once
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __syncthreads();
    constexpr int LPT = FI * 4, TPP = 64 / LPT, PASSES = 32 / TPP, AT_ONCE = PASSES < 4 ? PASSES : 4;
    float *reg = reinterpret_cast<float *>(lds) + wave * 32 * S::OUT_LD;
    const int lf = (lane % LPT) * 8;
    const int f = f0 + wf * FI * 32 + lf;
    const bool piece = SYM && nsteps != g.steps;
    // rows of X^T, of the mirrored tile, or of the output of a tall matrix
    const bool turned = EPI == APPLY || (SYM && ti != fi && !piece) || (EPI == LAST && g.tall);
    float df[8] = {};
    if (EPI == POLY && !piece && f < g.rows_w) {
        const float4 *d = reinterpret_cast<const float4 *>(g.d + static_cast<int64_t>(z) * g.rows_x + f);
        const float4 x = d[0], y = d[1];
        df[0] = x.x; df[1] = x.y; df[2] = x.z; df[3] = x.w;
        df[4] = y.x; df[5] = y.y; df[6] = y.z; df[7] = y.w;
    }
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
        const int tj = t0 + (wt * TJ + j) * 32;
        const bool there = tj < g.rows_x && f < g.rows_w;   // rows come in 64s: all 32 tokens or none
#pragma unroll
        for (int i = 0; i < FI; ++i)
#pragma unroll
            for (int r = 0; r < 16; r += 4)
                *reinterpret_cast<float4 *>(reg + (lane & 31) * S::OUT_LD + i * 32 + (r >> 2) * 8 + half * 4) =
                    make_float4(acc[i][j][r], acc[i][j][r + 1], acc[i][j][r + 2], acc[i][j][r + 3]);
        asm volatile("" ::: "memory");   // the accumulators' registers are free for what follows
        // four passes' operands at once: eight took registers that went to memory (B X of 4096 x 16384 643 -> 554 us)
#pragma unroll
        for (int p0 = 0; p0 < PASSES; p0 += AT_ONCE) {
            u32x4 hi[AT_ONCE], lo[AT_ONCE];   // of X, or O
            float et[AT_ONCE];                // the diagonal at the token
            if (there && EPI != GRAM && !piece) {
#pragma unroll
                for (int p = 0; p < AT_ONCE; ++p) {
                    const int t = tj + (p0 + p) * TPP + lane / LPT;
                    if constexpr (EPI == POLY) {
                        hi[p] = *reinterpret_cast<const u32x4 *>(g.o + z * g.ob + static_cast<int64_t>(t) * g.ldo + f);
                    } else {
                        const int64_t at = z * g.hb + static_cast<int64_t>(t) * g.ldh + f;
                        hi[p] = *reinterpret_cast<const u32x4 *>(g.hi + at);
                        lo[p] = *reinterpret_cast<const u32x4 *>(g.lo + at);
                    }
                    et[p] = (EPI == POLY ? g.d : g.e)[static_cast<int64_t>(z) * g.rows_x + t];
                }
            }
            __builtin_amdgcn_wave_barrier();
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            if (there) {
#pragma unroll
                for (int p = 0; p < AT_ONCE; ++p) {
                    const int tl = (p0 + p) * TPP + lane / LPT, t = tj + tl;
                    float *at = reg + tl * S::OUT_LD + lf;
                    const float4 x = reinterpret_cast<const float4 *>(at)[0], y = reinterpret_cast<const float4 *>(at)[1];
                    float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
                    if constexpr (SYM) {
                        if (piece) {
                            float4 *o = reinterpret_cast<float4 *>(
                                g.part + ((2ll * w + (kbeg == 0 ? 1 : 0)) * S::BT + (t - t0)) * S::BF + (f - f0));
                            o[0] = x;
                            o[1] = y;
                            continue;
                        }
                        symmetric_values<EPI>(g, z, t, f, hi[p], et[p], df, v);
                        symmetric_store<EPI>(g, z, t, f, v);
                    } else {
                        apply_values<EPI>(g, z, t, f, hi[p], lo[p], et[p], v);
                    }
                    if (turned) {
                        reinterpret_cast<float4 *>(at)[0] = make_float4(v[0], v[1], v[2], v[3]);
                        reinterpret_cast<float4 *>(at)[1] = make_float4(v[4], v[5], v[6], v[7]);
                    }
                }
            }
        }
        __builtin_amdgcn_wave_barrier();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (turned && tj < g.rows_x) {   // four lanes a feature, eight of its 32 tokens each
#pragma unroll 2
            for (int q = 0; q < FI * 2; ++q) {
                const int fl = q * 16 + (lane >> 2), tl = (lane & 3) * 8;
                const int64_t row = f0 + wf * FI * 32 + fl;
                if (row >= g.rows_w) continue;
                float v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) v[u] = reg[(tl + u) * S::OUT_LD + fl];
                turned_values<EPI>(g, z, row, tj + tl, v);
            }
        }
        __builtin_amdgcn_wave_barrier();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
    left -= nsteps;
    ++tile;
    s0 = 0;
    if (left > 0) __syncthreads();   // the sums are out of LDS before the next tile's operands come in
    }
}

// ---- small products ----------------------------------------------------------------------------
//
// Where the tiles above are few and short, a launch is their loads, barriers and chained instructions one
// after the other.  Here a workgroup takes 32 x 32 values, its eight waves an eighth of K each, straight
// from memory to the registers of the matrix instruction, all of it asked for at once up to K = 1024; the
// waves' sums meet in LDS and are added in wave order.  Over 221 random shapes it is the fastest for A A of 131
// (3 us of a call's five on average) and for B X of 35 (3 us).
constexpr int kFineWaves = 8;

template <int EPI>   // all but GRAM
__global__ __launch_bounds__(64 * kFineWaves, 2) void fine_kernel(Args g) {
    constexpr bool SYM = EPI == POLY;
    constexpr int U = 8, LD = 36;   // instructions' operands at once; floats between tokens
    __shared__ __attribute__((aligned(16))) float sums[kFineWaves][32 * LD];
    const int w = (blockIdx.x & 7) * g.per_xcd + (blockIdx.x >> 3);
    if (static_cast<int>(blockIdx.x >> 3) >= g.per_xcd || w >= g.total) return;
    const int z = w / g.per_batch, mn = w - z * g.per_batch;
    int ti, fi;
    if constexpr (SYM) {
        triangle(mn, ti, fi);
    } else {
        ti = mn / g.tiles_f;
        fi = mn - ti * g.tiles_f;
    }
    const int t0 = ti * 32, f0 = fi * 32, th = threadIdx.x, lane = th & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(th >> 6);
    // the finishing threads' operands: 128 threads, eight features of a token each
    const int t = t0 + (th >> 2), f = f0 + (th & 3) * 8;
    u32x4 hi = {0u, 0u, 0u, 0u};
    u32x4 lo = {0u, 0u, 0u, 0u};
    float et = 0.0f, df[8] = {};
    if (th < 128) {
        const int64_t row = static_cast<int64_t>(z) * g.rows_x;
        if constexpr (EPI == POLY) {
            hi = *reinterpret_cast<const u32x4 *>(g.o + z * g.ob + static_cast<int64_t>(t) * g.ldo + f);
            et = g.d[row + t];
#pragma unroll
            for (int u = 0; u < 8; ++u) df[u] = g.d[row + f + u];
        } else {
            const int64_t at = z * g.hb + static_cast<int64_t>(t) * g.ldh + f;
            hi = *reinterpret_cast<const u32x4 *>(g.hi + at);
            lo = *reinterpret_cast<const u32x4 *>(g.lo + at);
            et = g.e[row + t];
        }
    }
    const uint16_t *wrow = g.w + z * g.wb + static_cast<int64_t>(f0 + (lane & 31)) * g.ldw + half * 8;
    const uint16_t *xrow = g.x + z * g.xb + static_cast<int64_t>(t0 + (lane & 31)) * g.ldx + half * 8;
    const int total = g.steps * 4, total_x = SYM ? total : g.steps_x * 4;   // of 16 values of K
    const int beg = static_cast<int>(static_cast<int64_t>(total) * wave / kFineWaves);
    const int end = static_cast<int>(static_cast<int64_t>(total) * (wave + 1) / kFineWaves);
    auto fetch = [&](int s, h8 (&a)[U], h8 (&b)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u < end) {
                a[u] = *reinterpret_cast<const h8 *>(wrow + (s + u) * 16);
                b[u] = *reinterpret_cast<const h8 *>(xrow + (SYM || s + u < total_x ? s + u : s + u - total_x) * 16);
            }
        }
    };
    f16v acc[2] = {(f16v){}, (f16v){}};   // two chains
    auto use = [&](int s, h8 (&a)[U], h8 (&b)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s + u < end) acc[u & 1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[u], b[u], acc[u & 1], 0, 0, 0);
    };
    h8 a0[U], b0[U], a1[U], b1[U];
    fetch(beg, a0, b0);
    for (int s = beg; s < end; s += 2 * U) {
        fetch(s + U, a1, b1);
        use(s, a0, b0);
        fetch(s + 2 * U, a0, b0);
        use(s + U, a1, b1);
    }
#pragma unroll
    for (int r = 0; r < 16; r += 4)
        *reinterpret_cast<float4 *>(&sums[wave][(lane & 31) * LD + (r >> 2) * 8 + half * 4]) =
            make_float4(acc[0][r] + acc[1][r], acc[0][r + 1] + acc[1][r + 1], acc[0][r + 2] + acc[1][r + 2], acc[0][r + 3] + acc[1][r + 3]);
    __syncthreads();
    const bool turned = EPI == APPLY || (SYM && ti != fi) || (EPI == LAST && g.tall);
    if (th < 128) {
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        const int at = (th >> 2) * LD + (th & 3) * 8;
#pragma unroll
        for (int k = 0; k < kFineWaves; ++k) {
            const float4 x = *reinterpret_cast<const float4 *>(&sums[k][at]), y = *reinterpret_cast<const float4 *>(&sums[k][at + 4]);
            v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
            v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
        }
        if constexpr (SYM) {
            symmetric_values<EPI>(g, z, t, f, hi, et, df, v);
            symmetric_store<EPI>(g, z, t, f, v);
        } else {
            apply_values<EPI>(g, z, t, f, hi, lo, et, v);
        }
        if (turned) {   // each thread's own place of the first wave's sums
            *reinterpret_cast<float4 *>(&sums[0][at]) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(&sums[0][at + 4]) = make_float4(v[4], v[5], v[6], v[7]);
        }
    }
    if (!turned) return;
    __syncthreads();
    if (th < 128) {
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = sums[0][((th & 3) * 8 + u) * LD + (th >> 2)];
        turned_values<EPI>(g, z, f0 + (th >> 2), t0 + (th & 3) * 8, v);
    }
}

// Up to 64 rows, B is little work: every workgroup of B X forms the 32 rows of it that it needs, from O and
// its diagonal, in LDS, instead of a launch that forms it for all (64 x 64 54 -> 42 us, 48 with the rest of X;
// with 128 rows that takes longer than the launch, 16 x 128 x 512 71 -> 91).  A workgroup takes 32 rows of X and 256
// columns, 32 to a wave; everything that it reads is asked for at its start.
constexpr int kShortRows = 64;
constexpr int kShortCols = 256;

template <int EPI>   // APPLY or LAST
__global__ __launch_bounds__(512, 2) void apply_short_kernel(Args g) {
    constexpr int U = kShortRows / 16, LDB = kShortRows + 8, LD = 36;
    __shared__ __attribute__((aligned(16))) uint16_t b_rows[32 * LDB];
    __shared__ float diagonal[32];
    __shared__ __attribute__((aligned(16))) float sums[8][32 * LD];
    const int z = blockIdx.x / g.per_batch, mn = blockIdx.x - z * g.per_batch, ti = mn / g.tiles_f;
    const int th = threadIdx.x, lane = th & 63, half = lane >> 5, l32 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(th >> 6);
    const int t0 = ti * 32, f0 = (mn - ti * g.tiles_f) * kShortCols + wave * 32;
    const bool there = f0 < g.rows_w;   // of this wave's columns: all or none
    h8 a[U], rest[U];
    u32x4 hi[2], lo[2];
    if (there) {
        const uint16_t *row = g.w + z * g.wb + static_cast<int64_t>(f0 + l32) * g.ldw + half * 8;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            a[u] = *reinterpret_cast<const h8 *>(row + u * 16);
            rest[u] = *reinterpret_cast<const h8 *>(row + g.rest_at + u * 16);
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int64_t at = z * g.hb + static_cast<int64_t>(t0 + p * 16 + (lane >> 2)) * g.ldh + f0 + (lane & 3) * 8;
            hi[p] = *reinterpret_cast<const u32x4 *>(g.hi + at);
            lo[p] = *reinterpret_cast<const u32x4 *>(g.lo + at);
        }
    }
    if (wave * 32 < kShortRows) {   // columns 32 wave .. of B's rows t0 ..
        const uint16_t *o = g.o + z * g.ob;
        const float *d = g.d + static_cast<int64_t>(z) * g.rows_x;
        const int t = t0 + l32;
        h8 oc[U], ot[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            oc[u] = *reinterpret_cast<const h8 *>(o + static_cast<int64_t>(wave * 32 + l32) * g.ldo + u * 16 + half * 8);
            ot[u] = *reinterpret_cast<const h8 *>(o + static_cast<int64_t>(t) * g.ldo + u * 16 + half * 8);
        }
        const float dt = d[t];
        uint2 here[4];
        float4 df[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int c = wave * 32 + r * 8 + half * 4;
            here[r] = *reinterpret_cast<const uint2 *>(o + static_cast<int64_t>(t) * g.ldo + c);
            df[r] = *reinterpret_cast<const float4 *>(d + c);
        }
        f16v sum = {};
#pragma unroll
        for (int u = 0; u < U; ++u)
            sum = __builtin_amdgcn_mfma_f32_32x32x16_f16(oc[u], ot[u], sum, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int c = wave * 32 + r * 8 + half * 4;
            const h4 o4 = __builtin_bit_cast(h4, here[r]);
            const float dc[4] = {df[r].x, df[r].y, df[r].z, df[r].w};
            h4 b;
#pragma unroll
            for (int u = 0; u < 4; ++u) {   // symmetric_values<POLY>
                const float ov = static_cast<float>(o4[u]) * g.inv_o;
                float square = fmaf(dt + dc[u], ov, sum[r * 4 + u] * g.inv_poly);
                float v = fmaf(g.c, square, g.b * ov) * g.sb;
                if (t == c + u) {
                    square = fmaf(dt, dt, square);
                    diagonal[l32] = g.a + fmaf(g.c, square, g.b * dt);
                    v = 0.0f;
                }
                b[u] = static_cast<_Float16>(v);
            }
            *reinterpret_cast<uint2 *>(b_rows + l32 * LDB + c) = __builtin_bit_cast(uint2, b);
        }
    }
    __syncthreads();
    if (!there) return;
    f16v acc = {};
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const h8 b = *reinterpret_cast<const h8 *>(b_rows + l32 * LDB + u * 16 + half * 8);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[u], b, acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(rest[u], b, acc, 0, 0, 0);
    }
    float *reg = sums[wave];   // this wave's alone
#pragma unroll
    for (int r = 0; r < 16; r += 4)
        *reinterpret_cast<float4 *>(reg + l32 * LD + (r >> 2) * 8 + half * 4) = make_float4(acc[r], acc[r + 1], acc[r + 2], acc[r + 3]);
    __builtin_amdgcn_wave_barrier();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const bool turned = EPI == APPLY || g.tall;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int tl = p * 16 + (lane >> 2), at = tl * LD + (lane & 3) * 8;
        const float4 x = *reinterpret_cast<const float4 *>(reg + at), y = *reinterpret_cast<const float4 *>(reg + at + 4);
        float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        apply_values<EPI>(g, z, t0 + tl, f0 + (lane & 3) * 8, hi[p], lo[p], diagonal[tl], v);
        if (turned) {
            *reinterpret_cast<float4 *>(reg + at) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(reg + at + 4) = make_float4(v[4], v[5], v[6], v[7]);
        }
    }
    if (!turned) return;
    __builtin_amdgcn_wave_barrier();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int fl = q * 16 + (lane >> 2), tl = (lane & 3) * 8;
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = reg[(tl + u) * LD + fl];
        turned_values<EPI>(g, z, f0 + fl, t0 + tl, v);
    }
}

// Adds pieces k .. k + N - 1, up to the last, to v; all of their loads are under way at once.  The first one ends
// its range, the others start theirs.
template <int N>
__device__ __forceinline__ int add_pieces(const float *p, int size, int first, int k, int last, float (&v)[4]) {
    float4 x[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const int i = min(k + u, last);
        x[u] = *reinterpret_cast<const float4 *>(p + static_cast<int64_t>(2 * i + (i == first ? 1 : 0)) * size);
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const bool in = k + u <= last;   // a choice and no branch, or each load moves behind one
        const float q[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = in ? v[e] + q[e] : v[e];
    }
    return N;
}

// The pieces of X X^T's tiles that more than one workgroup had, added in the order of their steps, 16 x 64
// values a workgroup (few tiles have many pieces each, and a thread's chain of loads is the launch's time: 64 x
// 12000, with 47 pieces of its one tile, 11.3 us with 64 x 64 a workgroup, 4.6 so), stored as they are and, off the diagonal, transposed.
constexpr int kFoldRows = 16;
template <int SIDE>
__global__ __launch_bounds__(256) void fold_kernel(Args g) {
    constexpr int ACROSS = SIDE / 64, PARTS = ACROSS * (SIDE / kFoldRows);
    __shared__ float turn[kFoldRows][65];
    const int tile = blockIdx.x / PARTS, part = blockIdx.x % PARTS, th = threadIdx.x;
    const int64_t units = static_cast<int64_t>(g.total) * g.steps, from = static_cast<int64_t>(tile) * g.steps;
    // the last range that starts at or before a unit u is ceil((u + 1) groups / units) - 1
    auto owner = [&](int64_t u) { return static_cast<int>(((u + 1) * g.groups + units - 1) / units) - 1; };
    const int first = owner(from), last = owner(from + g.steps - 1);
    if (first == last) return;
    const int z = tile / g.per_batch;
    int ti, fi;
    triangle(tile - z * g.per_batch, ti, fi);
    const int tp = part / ACROSS * kFoldRows, fp = part % ACROSS * 64, t0 = ti * SIDE + tp, f0 = fi * SIDE + fp;
    if (t0 >= g.rows_x || f0 >= g.rows_w) return;   // rows come in 64s
    const int tl = th >> 4, fl = (th & 15) * 4, t = t0 + tl, f = f0 + fl;
    float v[4] = {};
    const float *p = g.part + static_cast<int64_t>(tp + tl) * SIDE + fp + fl;
    int k = first;
    while (last - k >= 4) k += add_pieces<24>(p, SIDE * SIDE, first, k, last, v);
    if (k <= last) add_pieces<4>(p, SIDE * SIDE, first, k, last, v);
    gram_values(g, z, t, f, v);
    *reinterpret_cast<uint2 *>(g.o + z * g.ob + static_cast<int64_t>(t) * g.ldo + f) = pack_h4(v);
    if (ti == fi) return;
#pragma unroll
    for (int u = 0; u < 4; ++u) turn[tl][fl + u] = v[u];
    __syncthreads();
    const int row = th >> 2, from_t = (th & 3) * 4;
    float w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) w[u] = turn[from_t + u][row];
    *reinterpret_cast<uint2 *>(g.o + z * g.ob + static_cast<int64_t>(f0 + row) * g.ldo + t0 + from_t) = pack_h4(w);
}

// ---- plan and launches ---------------------------------------------------------------------------

using Big = linear::Shape<256, 256, 2, 4, 3, 2>;        // one workgroup of eight waves per CU
using Mid = linear::Shape<128, 128, 2, 2, 3, 2>;        // two of four
using Small = linear::Shape<64, 64, 2, 2, 4, 4>;        // two of four
using MidDeep = linear::Shape<128, 128, 2, 2, 5, 4>;    // one of four, with more steps in flight
static_assert(kSide[BIG] == Big::BF && kSide[MID] == Mid::BF && kSide[SMALL] == Small::BF && kSide[MID_DEEP] == MidDeep::BF &&
              kPerCu[BIG] == Big::PER_CU && kPerCu[MID] == Mid::PER_CU && kPerCu[SMALL] == Small::PER_CU && kPerCu[MID_DEEP] == MidDeep::PER_CU,
              "the plan's tiles are the kernels'");

size_t piece_bytes(const Plan &p) {
    return p.groups == p.total ? 0 : static_cast<size_t>(p.groups) * 2 * kSide[p.shape] * kSide[p.shape] * 4;
}

struct Layout {
    int64_t r, c, rp, cp, ldx, ldt, ldr;   // ldx: of X; ldt: of X^T; ldr: of O, B
    Plan gram, poly, apply;
    size_t off_hi, off_lo, off_t0, off_t1, off_o, off_b, off_d, off_e, off_norm, off_part, bytes;
};
// Rows that lie a multiple of 4 KB apart meet in few of the caches' sets (8% of a product): 128 bytes more.
int64_t apart(int64_t padded) { return padded * 2 % 4096 == 0 ? padded + kUnit : padded; }
Layout layout(int64_t batch, int64_t rows, int64_t cols, bool rest) {
    Layout L;
    L.r = std::min(rows, cols);
    L.c = std::max(rows, cols);
    L.rp = round_up(L.r, kUnit);
    L.cp = round_up(L.c, kUnit);
    L.ldx = apart(L.cp);
    L.ldt = apart(rest ? 2 * L.rp : L.rp);
    L.ldr = apart(L.rp);
    L.gram = plan_of(batch, L.rp, L.rp, L.cp / kUnit, true, true);
    L.poly = plan_of(batch, L.rp, L.rp, L.rp / kUnit, true, false);
    L.apply = plan_of(batch, L.rp, L.cp, (rest ? 2 : 1) * L.rp / kUnit, false, false);
    const size_t x = align256(static_cast<size_t>(batch) * L.rp * L.ldx * 2), t = align256(static_cast<size_t>(batch) * L.cp * L.ldt * 2);
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
    o += piece_bytes(L.gram);
    L.bytes = o;
    return L;
}

template <class S, int EPI>
hipError_t launch_tiles(const Args &g, hipStream_t st) {
    hipLaunchKernelGGL((ortho_kernel<S, EPI>), dim3(static_cast<unsigned>(g.per_xcd) * 8u), dim3(64 * S::NW), 0, st, g);
    if constexpr (EPI == GRAM) {
        if (g.groups != g.total) {
            hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            constexpr int parts = S::BF / 64 * (S::BF / kFoldRows);
            hipLaunchKernelGGL((fold_kernel<S::BF>), dim3(static_cast<unsigned>(g.total) * parts), dim3(256), 0, st, g);
        }
    }
    return hipGetLastError();
}
template <int EPI>
hipError_t launch_product(Args g, const Plan &p, hipStream_t st) {
    g.groups = p.groups;
    g.per_batch = static_cast<int>(p.tiles);
    g.total = static_cast<int>(p.total);
    g.tiles_f = static_cast<int>(ceil_div(g.rows_w, kSide[p.shape]));
    g.per_xcd = static_cast<int>(ceil_div(g.groups, 8));
    switch (p.shape) {
        case BIG: return launch_tiles<Big, EPI>(g, st);
        case MID: return launch_tiles<Mid, EPI>(g, st);
        case MID_DEEP: return launch_tiles<MidDeep, EPI>(g, st);
        case FINE:
            if constexpr (EPI == GRAM) return hipErrorInvalidValue;   // not planned
            else hipLaunchKernelGGL((fine_kernel<EPI>), dim3(static_cast<unsigned>(g.per_xcd) * 8u), dim3(64 * kFineWaves), 0, st, g);
            return hipGetLastError();
        default: return launch_tiles<Small, EPI>(g, st);
    }
}

}  // namespace

size_t orthogonalise_workspace_bytes(int64_t batch, int64_t rows, int64_t cols) {
    return batch > 0 ? layout(batch, rows, cols, true).bytes : 0;   // whatever the steps and coefficients
}

hipError_t launch_orthogonalise(const OrthoArgs &a, hipStream_t st) {
    if (a.batch <= 0) return hipSuccess;
    const Powers sc = powers_of(std::min(a.rows, a.cols), a.steps, a.a, a.b, a.c);
    if (!sc.fit) return hipErrorInvalidValue;
    const Layout L = layout(a.batch, a.rows, a.cols, sc.rest);
    char *ws = static_cast<char *>(a.workspace);
    auto half = [&](size_t off) { return reinterpret_cast<uint16_t *>(ws + off); };
    const int tall = a.rows > a.cols;
    const float s = sc.x;

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
    l.ldt = L.ldt;
    l.xb = L.rp * L.ldx;
    l.tb = L.cp * L.ldt;
    l.rest_at = sc.rest ? static_cast<int>(L.rp) : 0;
    l.rp = static_cast<int>(L.rp);
    l.cp = static_cast<int>(L.cp);
    l.tall = tall;
    l.s = s;
    l.eps = a.eps;
    // a workgroup a piece of 2048 values, up to 1024 of them a matrix and about as many for a batch
    const int64_t pieces = a.rows * ceil_div(a.cols, 2048);
    l.groups = static_cast<int>(std::min(pieces, std::max<int64_t>(64, kNormGroups / a.batch)));
    const dim3 norm_grid(static_cast<unsigned>(l.groups), static_cast<unsigned>(a.batch));
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
    g.rest_at = l.rest_at;
    g.so = sc.o;
    g.sb = sc.b;
    g.inv_o = 1.0f / sc.o;
    g.inv_b = 1.0f / sc.b;
    g.ldh = L.ldx;
    g.hb = l.xb;
    g.ldt = L.ldt;
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
        if ((e = launch_product<GRAM>(g, L.gram, st)) != hipSuccess) return e;
        if (L.rp <= kShortRows) {
            g.w = half(k & 1 ? L.off_t1 : L.off_t0);
            g.ldw = L.ldt;
            g.wb = l.tb;
            g.xt = half(k & 1 ? L.off_t0 : L.off_t1);
            g.rows_w = static_cast<int>(L.cp);
            g.inv = 1.0f / s;
            g.inv_poly = g.inv_o * g.inv_o;
            g.tiles_f = static_cast<int>(ceil_div(L.cp, kShortCols));
            g.per_batch = static_cast<int>(L.rp / 32) * g.tiles_f;
            const dim3 grid(static_cast<unsigned>(g.per_batch * a.batch));
            if (k + 1 < a.steps) hipLaunchKernelGGL((apply_short_kernel<APPLY>), grid, dim3(512), 0, st, g);
            else hipLaunchKernelGGL((apply_short_kernel<LAST>), grid, dim3(512), 0, st, g);
            if ((e = hipGetLastError()) != hipSuccess) return e;
            continue;
        }
        g.w = g.x = g.o;
        g.ldw = g.ldx = L.ldr;
        g.wb = g.xb = g.ob;
        g.steps = static_cast<int>(L.rp / kUnit);
        g.inv = g.inv_o * g.inv_o;
        if ((e = launch_product<POLY>(g, L.poly, st)) != hipSuccess) return e;
        g.x = g.bo;
        g.w = half(k & 1 ? L.off_t1 : L.off_t0);
        g.xt = half(k & 1 ? L.off_t0 : L.off_t1);
        g.ldw = L.ldt;
        g.wb = l.tb;
        g.rows_w = static_cast<int>(L.cp);
        g.steps_x = g.steps;
        if (sc.rest) g.steps *= 2;
        g.inv = 1.0f / s;
        e = k + 1 < a.steps ? launch_product<APPLY>(g, L.apply, st) : launch_product<LAST>(g, L.apply, st);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace lce
