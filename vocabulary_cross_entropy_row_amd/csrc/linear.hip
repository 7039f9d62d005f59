// Matrix product with bias, activation and residual in its epilogue, and its
// backward (linear_mfma.h has the kernel).
//
// Forward: one launch, or with K split over workgroups (few tiles) a second one
// that adds the partial sums in their order and runs the epilogue.
//
// Backward, with dz = grad_out act'(z):
//   grad_x = dz W        the same kernel on dz [n, M] and W^T [K, M]
//   grad_W = dz^T x      ... on dz^T [M, n] and x^T [K, n]
//   grad_b = sum dz      column sums, fp32 partials per 128 rows folded in order
// One launch reads grad_out (and the pre-activation), the weight and x, and writes dz,
// dz^T, the bias's partial sums, W^T and x^T.
#include <hip/hip_runtime.h>
#include <algorithm>
#include <stdint.h>

#include "ce_device.h"
#include "head_internal.h"
#include "linear_mfma.h"
#include "linear_plan.h"

namespace lce {
namespace {

using dev::Elt;
using dev::u32x4;

using linear_plan::ceil_div;
using linear_plan::round_up;
size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
bool on16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// ---- tile shapes ------------------------------------------------------------------

using Big = linear::Shape<256, 256, 2, 4, 3, 2>;    // one workgroup of eight waves per CU
using Wide = linear::Shape<256, 128, 4, 2, 3, 3>;   // one
using Low = linear::Shape<128, 64, 2, 2, 3, 3>;     // two of four waves
using Tiny = linear::Shape<64, 32, 2, 1, 4, 4>;     // three of two
using namespace linear_plan;

template <class S>
constexpr bool planned(int i) {
    return kShapes[i].bf == S::BF && kShapes[i].bt == S::BT && kShapes[i].threads == 64 * S::NW;
}
static_assert(planned<Big>(BIG) && planned<Wide>(WIDE) && planned<Low>(LOW) && planned<Tiny>(TINY) &&
              kShapes[ROWS16].threads == 64 * linear::kRowsWaves && kShapes[ROWS32].threads == 64 * linear::kRowsWaves,
              "the plan's tiles are the kernels'");

constexpr int64_t kLastCache = int64_t(256) << 20;   // bytes of the cache in front of HBM

template <class S>
hipError_t launch_shape(const linear::Args &g, bool fp8, hipStream_t st) {
    const dim3 grid(static_cast<unsigned>(g.per_xcd) * 8u), block(64 * S::NW);
    const bool tail = g.kbytes % linear::kStep != 0;
    if (fp8) {
        if (tail) hipLaunchKernelGGL((linear::linear_kernel<S, true, true>), grid, block, 0, st, g);
        else hipLaunchKernelGGL((linear::linear_kernel<S, true, false>), grid, block, 0, st, g);
    } else {
        if (tail) hipLaunchKernelGGL((linear::linear_kernel<S, false, true>), grid, block, 0, st, g);
        else hipLaunchKernelGGL((linear::linear_kernel<S, false, false>), grid, block, 0, st, g);
    }
    return hipGetLastError();
}
template <int TT>
hipError_t launch_rows(const linear::Args &g, bool fp8, hipStream_t st) {
    const dim3 grid(static_cast<unsigned>(ceil_div(g.M, 16))), block(64 * linear::kRowsWaves);
    if (fp8) hipLaunchKernelGGL((linear::linear_rows_kernel<true, TT>), grid, block, 0, st, g);
    else hipLaunchKernelGGL((linear::linear_rows_kernel<false, TT>), grid, block, 0, st, g);
    return hipGetLastError();
}

// ---- what the backward's products read ---------------------------------------------------

constexpr int kTrRows = 128, kTrCols = 64;

// One matrix to transpose: v = in, or in act'(pre); out[r][c] = bf16(v) when out is given; out_t[c][r] =
// bf16(v), rows [rows, rows_pad) as zeros; sums of v, not rounded, over the rows of a block of 128, to
// part[block][c], or to `total` where there is one block only.
struct Transpose {
    const void *in;        // [rows, cols] bf16 or fp32
    int64_t ld_in;
    const uint16_t *pre;   // bf16, or NULL
    int64_t ld_pre;
    int act;
    uint16_t *out;         // [rows, cols] or NULL
    int64_t ld_out;
    uint16_t *out_t;       // [cols, rows_pad] or NULL
    int64_t ld_t;
    float *part;           // [row blocks][cols] or NULL
    void *total;           // [cols] bf16 or fp32, or NULL
    int rows, rows_pad, cols;
    int tiles_c;           // column tiles
    bool in_bf16, total_bf16;
};
constexpr int kMaxJobs = 3;
struct TransposeJobs {
    Transpose job[kMaxJobs];
    unsigned end[kMaxJobs];   // one past the job's last workgroup
};
// All the transposes of a backward in one launch.  A tile of 128 x 64 goes through LDS, 16-byte chunk c
// of row r at c ^ (r / 8 mod 8): the writes of a wave cover 1 KB without conflicts and the eight rows
// of an output chunk are read from different banks.  Bound by memory (4096 x 16384 with an activation,
// its weight and its input of width 4096, 870 MB: 170 us).
__global__ __launch_bounds__(256) void transpose_kernel(TransposeJobs jobs) {
    constexpr int PER = kTrRows * (kTrCols / 8) / 256;   // 16-byte chunks per thread
    __shared__ __align__(16) uint16_t tile[kTrRows * kTrCols];
    __shared__ float sums[32][kTrCols];   // per row of threads
    const unsigned b = blockIdx.x;
    const int j = b < jobs.end[0] ? 0 : (b < jobs.end[1] ? 1 : 2);
    const Transpose &a = jobs.job[j];
    const int tile_at = static_cast<int>(b - (j ? jobs.end[j - 1] : 0));
    const int block = tile_at / a.tiles_c;
    float sum[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    const int r0 = block * kTrRows, c0 = (tile_at - block * a.tiles_c) * kTrCols;
    const int t = threadIdx.x;
#pragma unroll
    for (int h = 0; h < PER; ++h) {
        const int idx = t + h * 256, r = idx >> 3, ch = idx & 7;
        const int gr = r0 + r, gc = c0 + ch * 8;
        const bool full = gr < a.rows && gc + 8 <= a.cols;
        float v[8];
        if (full && a.in_bf16) {
            const u32x4 q = *reinterpret_cast<const linear::any16 *>(static_cast<const uint16_t *>(a.in) + gr * a.ld_in + gc);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = Elt<true>::get(q, e);
        } else if (full) {
            const linear::any16 *q = reinterpret_cast<const linear::any16 *>(static_cast<const float *>(a.in) + gr * a.ld_in + gc);
            const u32x4 x = q[0], y = q[1];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = Elt<false>::get(e < 4 ? x : y, e & 3);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = gr >= a.rows || gc + e >= a.cols ? 0.0f
                       : a.in_bf16                      ? Elt<true>::load_one(a.in, gr * a.ld_in + gc + e)
                                                        : Elt<false>::load_one(a.in, gr * a.ld_in + gc + e);
        }
        if (a.pre) {
            float z[8];
            if (full) {
                const u32x4 q = *reinterpret_cast<const linear::any16 *>(a.pre + gr * a.ld_pre + gc);
#pragma unroll
                for (int e = 0; e < 8; ++e) z[e] = Elt<true>::get(q, e);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    z[e] = gr < a.rows && gc + e < a.cols ? Elt<true>::load_one(a.pre, gr * a.ld_pre + gc + e) : 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = gr < a.rows && gc + e < a.cols ? v[e] * linear::slope(a.act, z[e]) : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += v[e];   // a thread's chunks are of the same eight columns
        const u32x4 q = Elt<true>::pack(v);
        if (a.out) {   // ld_out and out are 16-byte whole
            if (full) {
                *reinterpret_cast<u32x4 *>(a.out + gr * a.ld_out + gc) = q;
            } else if (gr < a.rows) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (gc + e < a.cols) Elt<true>::store_one(a.out, gr * a.ld_out + gc + e, v[e]);
            }
        }
        *reinterpret_cast<u32x4 *>(tile + r * kTrCols + ((ch ^ (r >> 3)) & 7) * 8) = q;
    }
    const bool summed = a.part || a.total;
    if (summed) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[t >> 3][(t & 7) * 8 + e] = sum[e];
    }
    __syncthreads();
    if (a.out_t) {
#pragma unroll
        for (int h = 0; h < PER; ++h) {
            const int idx = t + h * 256;
            const int orow = (idx >> 3) & 63, ch = (idx & 7) + 8 * (idx >> 9);
            const int gc = c0 + orow, gr = r0 + ch * 8;
            if (gc >= a.cols || gr >= a.rows_pad) continue;   // rows_pad is a multiple of 8
            const uint16_t *src = tile + ch * 8 * kTrCols + (((orow >> 3) ^ ch) & 7) * 8 + (orow & 7);
            u32x4 o;
#pragma unroll
            for (int w = 0; w < 4; ++w)
                o[w] = src[2 * w * kTrCols] | (static_cast<uint32_t>(src[(2 * w + 1) * kTrCols]) << 16);
            *reinterpret_cast<u32x4 *>(a.out_t + gc * a.ld_t + gr) = o;
        }
    }
    if (summed && t < kTrCols && c0 + t < a.cols) {
        float v = sums[0][t];
        for (int r = 1; r < 32; ++r) v += sums[r][t];
        if (a.part) a.part[static_cast<int64_t>(block) * a.cols + c0 + t] = v;
        else if (a.total_bf16) Elt<true>::store_one(a.total, c0 + t, v);
        else static_cast<float *>(a.total)[c0 + t] = v;
    }
}

// Workspace of the backward: regions in bytes
struct GradLayout {
    int64_t np;   // tokens in whole eights
    size_t off_dz, off_dzt, off_xt, off_wt, off_bias, off_part, bytes;
};
GradLayout grad_layout(int64_t n, int64_t K, int64_t M) {
    GradLayout L;
    L.np = round_up(n, 8);
    size_t o = 0;
    L.off_dz = o;    o += align256(static_cast<size_t>(n) * M * 2);
    L.off_dzt = o;   o += align256(static_cast<size_t>(L.np) * M * 2);
    L.off_xt = o;    o += align256(static_cast<size_t>(L.np) * K * 2);
    L.off_wt = o;    o += align256(static_cast<size_t>(M) * K * 2);
    L.off_bias = o;  o += align256(static_cast<size_t>(ceil_div(n, kTrRows)) * M * 4);
    L.off_part = o;
    o += align256(std::max(linear_workspace_bytes(n, M, K, false), linear_workspace_bytes(M, L.np, K, false)));
    L.bytes = o;
    return L;
}

}  // namespace

size_t linear_workspace_bytes(int64_t n, int64_t K, int64_t M, bool fp8) {
    if (n <= 0 || M <= 0) return 0;
    const Plan p = plan_of(n, K, M, fp8);
    return p.splits > 1 ? static_cast<size_t>(p.splits) * n * round_up(M, 8) * 4 : 0;
}

hipError_t launch_linear(const LinearArgs &a, hipStream_t st) {
    if (a.n <= 0 || a.M <= 0) return hipSuccess;
    const int es = a.fp8 ? 1 : 2;
    const Plan p = plan_of(a.n, a.K, a.M, a.fp8);
    const ShapeInfo &s = kShapes[p.shape];
    linear::Args g;
    g.w = static_cast<const unsigned char *>(a.weight);
    g.x = static_cast<const unsigned char *>(a.x);
    g.ldw = a.ldw * es;
    g.ldx = a.ldx * es;
    g.kbytes = static_cast<int>(a.K * es);
    g.n = static_cast<int>(a.n);
    g.M = static_cast<int>(a.M);
    const int64_t tf = ceil_div(a.M, s.bf), tt = ceil_div(a.n, s.bt), total = tf * tt * p.splits;
    if (round_up(total, 8) * s.threads > kMaxThreads) return hipErrorInvalidValue;   // outputs past the card's memory
    g.tiles_f = static_cast<int>(tf);
    g.tiles_t = static_cast<int>(tt);
    g.splits = p.splits;
    g.per_xcd = static_cast<int>(ceil_div(total, 8));
    g.part = a.part;
    g.ldpart = round_up(a.M, 8);
    linear::Epi &e = g.e;
    e.scale_x = a.scale_x;
    e.scale_w = a.scale_w;
    e.bias = a.bias;
    e.bias_bf16 = a.bias_bf16;
    e.act = a.act;
    e.residual = a.residual;
    e.ldr = a.ldr;
    e.out = a.out;
    e.ldo = a.ldo;
    e.out_bf16 = a.out_bf16;
    // An output that the last cache cannot hold for its reader need not displace the operands there:
    // 4096 x 1024 x 65536 575 -> 530 us and with the cross-entropy that reads it 773 -> 725, 16384 x 512 x
    // 32000 728 -> 635 and 1102 -> 985, 4096 x 1024 x 50256 e4m3 314 -> 290.  Smaller ones would cost their
    // reader more than the product gains (4096 x 1024 x 32768 and the cross-entropy 353 -> 364), rows that
    // start inside 16 bytes write parts of lines (4096 x 4096 x 50257 1366 -> 1400), and so do fp32 ones
    // (4096 x 1024 x 32768 331 -> 374).
    e.streams = a.out_bf16 && a.n * a.M * 2 > kLastCache && on16(a.out) && a.ldo % 8 == 0;
    e.preact = a.preact;
    e.ldp = a.ldp;
    e.n = a.n;
    e.M = a.M;
    hipError_t err;
    switch (p.shape) {
        case BIG: err = launch_shape<Big>(g, a.fp8, st); break;
        case WIDE: err = launch_shape<Wide>(g, a.fp8, st); break;
        case LOW: err = launch_shape<Low>(g, a.fp8, st); break;
        case TINY: err = launch_shape<Tiny>(g, a.fp8, st); break;
        case ROWS16: err = launch_rows<1>(g, a.fp8, st); break;
        default: err = launch_rows<2>(g, a.fp8, st); break;
    }
    if (err != hipSuccess || p.splits == 1) return err;
    const int64_t items = a.n * (g.ldpart / 8);
    hipLaunchKernelGGL(linear::linear_fold_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(ceil_div(items, 256), 16384))),
                       dim3(256), 0, st, a.part, g.ldpart, p.splits, e);
    return hipGetLastError();
}

size_t linear_backward_workspace_bytes(int64_t n, int64_t K, int64_t M) { return grad_layout(n, K, M).bytes; }

hipError_t launch_linear_backward(const LinearGradArgs &a, hipStream_t st) {
    const GradLayout L = grad_layout(a.n, a.K, a.M);
    char *ws = static_cast<char *>(a.workspace);
    uint16_t *dz = reinterpret_cast<uint16_t *>(ws + L.off_dz), *dzt = reinterpret_cast<uint16_t *>(ws + L.off_dzt);
    uint16_t *xt = reinterpret_cast<uint16_t *>(ws + L.off_xt), *wt = reinterpret_cast<uint16_t *>(ws + L.off_wt);
    float *bias_part = reinterpret_cast<float *>(ws + L.off_bias), *part = reinterpret_cast<float *>(ws + L.off_part);
    const bool active = a.act != ACT_NONE;
    // without an activation a bf16 grad_out whose rows the product can read, and does not overwrite, is dz
    const bool direct = !active && a.grad_bf16 && on16(a.grad_out) && a.ldg % 8 == 0 &&
                        a.ldg <= kLinearMaxStride / 2 && a.grad_out != a.grad_x;
    hipError_t e;
    TransposeJobs jobs{};
    int count = 0;
    unsigned groups = 0;
    auto add = [&](const Transpose &t) {
        jobs.job[count] = t;
        jobs.job[count].tiles_c = static_cast<int>(ceil_div(t.cols, kTrCols));
        groups += static_cast<unsigned>(ceil_div(t.cols, kTrCols) * ceil_div(std::max(t.rows, t.rows_pad), kTrRows));
        jobs.end[count++] = groups;
    };
    const bool one_block = a.n > 0 && a.n <= kTrRows;   // its column sums are the bias's gradient
    Transpose d{};
    d.in = a.grad_out;
    d.ld_in = a.ldg;
    d.in_bf16 = a.grad_bf16;
    d.pre = active ? static_cast<const uint16_t *>(a.preact) : nullptr;
    d.ld_pre = a.ldp;
    d.act = a.act;
    d.out = a.grad_x && !direct ? dz : nullptr;
    d.ld_out = a.M;
    d.out_t = a.grad_weight ? dzt : nullptr;
    d.ld_t = L.np;
    d.part = a.grad_bias && !one_block ? bias_part : nullptr;
    d.total = one_block ? a.grad_bias : nullptr;
    d.total_bf16 = a.grad_bias_bf16;
    d.rows = static_cast<int>(a.n);
    d.rows_pad = static_cast<int>(L.np);
    d.cols = static_cast<int>(a.M);
    if (a.n > 0 && (d.out || d.out_t || d.part || d.total)) add(d);
    if (a.grad_x && a.n > 0) {   // W^T
        Transpose t{};
        t.in = a.weight;
        t.ld_in = a.ldw;
        t.in_bf16 = true;
        t.out_t = wt;
        t.ld_t = a.M;
        t.rows = t.rows_pad = static_cast<int>(a.M);
        t.cols = static_cast<int>(a.K);
        add(t);
    }
    if (a.grad_weight && a.n > 0) {   // x^T
        Transpose t{};
        t.in = a.x;
        t.ld_in = a.ldx;
        t.in_bf16 = true;
        t.out_t = xt;
        t.ld_t = L.np;
        t.rows = static_cast<int>(a.n);
        t.rows_pad = static_cast<int>(L.np);
        t.cols = static_cast<int>(a.K);
        add(t);
    }
    for (int j = count; j < kMaxJobs; ++j) jobs.end[j] = groups;
    if (groups) {
        hipLaunchKernelGGL(transpose_kernel, dim3(groups), dim3(256), 0, st, jobs);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (a.grad_bias && !one_block &&
        (e = launch_column_fold(bias_part, ceil_div(a.n, kTrRows), a.M, a.M, a.grad_bias, a.grad_bias_bf16, st)) != hipSuccess)
        return e;
    if (a.grad_x && a.n > 0) {
        LinearArgs g{};
        g.x = direct ? a.grad_out : dz;
        g.ldx = direct ? a.ldg : a.M;
        g.weight = wt;
        g.ldw = a.M;
        g.n = a.n;
        g.K = a.M;
        g.M = a.K;
        g.out = a.grad_x;
        g.ldo = a.ldgx;
        g.out_bf16 = true;
        g.part = part;
        if ((e = launch_linear(g, st)) != hipSuccess) return e;
    }
    if (a.grad_weight) {
        LinearArgs g{};
        g.x = dzt;
        g.ldx = L.np;
        g.weight = xt;
        g.ldw = L.np;
        g.n = a.M;
        g.K = L.np;
        g.M = a.K;
        g.out = a.grad_weight;
        g.ldo = a.K;
        g.out_bf16 = a.grad_weight_bf16;
        g.part = part;
        if ((e = launch_linear(g, st)) != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace lce
