// Matrix product of e4m3 operands with a scale for each block of 128 (blocks_mfma.h has the kernels), and
// the backward of its training form:
//   grad_x = Qrow(g) W      g [n, M] in row blocks, W^T [K, M] in tiles
//   grad_W = Qrow(g^T) x    g^T [M, n] in row blocks, x^T [K, n] in tiles
//   grad_b = sum g          column sums, fp32 partials per 128 rows folded in order
// One launch reads grad_out and writes both of its quantised forms and the bias's partial sums.
#include <hip/hip_runtime.h>
#include <algorithm>
#include <stdint.h>

#include "blocks_internal.h"
#include "blocks_mfma.h"
#include "head_internal.h"
#include "blocks_plan.h"

namespace lce {
namespace {

using namespace blocks_plan;
size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

using Big = linear::Shape<256, 256, 2, 4, 3, 2>;
using Wide = linear::Shape<256, 128, 4, 2, 3, 2>;
using Low = linear::Shape<128, 64, 2, 2, 3, 2>;
using Tiny = linear::Shape<64, 32, 2, 1, 4, 3>;

template <class S>
constexpr bool planned(int i) {
    return kShapes[i].bf == S::BF && kShapes[i].bt == S::BT && kShapes[i].threads == 64 * S::NW && kShapes[i].per_cu == S::PER_CU;
}
static_assert(planned<Big>(BIG) && planned<Wide>(WIDE) && planned<Low>(LOW) && planned<Tiny>(TINY) &&
              kShapes[ROWS16].threads == 64 * blocks::kRowsWaves && kShapes[ROWS32].threads == 64 * blocks::kRowsWaves,
              "the plan's tiles are the kernels'");

template <class S>
hipError_t launch_shape(const blocks::Args &g, bool pow2, hipStream_t st) {
    const dim3 grid(static_cast<unsigned>(g.per_xcd) * 8u), block(64 * S::NW);
    if (pow2) hipLaunchKernelGGL((blocks::blocks_kernel<S, true>), grid, block, 0, st, g);
    else hipLaunchKernelGGL((blocks::blocks_kernel<S, false>), grid, block, 0, st, g);
    return hipGetLastError();
}
template <int TT>
hipError_t launch_rows(const blocks::Args &g, bool pow2, hipStream_t st) {
    const dim3 grid(static_cast<unsigned>(ceil_div(g.M, 16))), block(64 * blocks::kRowsWaves);
    const bool cut = g.K % 16 != 0;
    if (pow2) {
        if (cut) hipLaunchKernelGGL((blocks::blocks_rows_kernel<true, true, TT>), grid, block, 0, st, g);
        else hipLaunchKernelGGL((blocks::blocks_rows_kernel<true, false, TT>), grid, block, 0, st, g);
    } else {
        if (cut) hipLaunchKernelGGL((blocks::blocks_rows_kernel<false, true, TT>), grid, block, 0, st, g);
        else hipLaunchKernelGGL((blocks::blocks_rows_kernel<false, false, TT>), grid, block, 0, st, g);
    }
    return hipGetLastError();
}

__global__ __launch_bounds__(256) void zero_kernel(uint16_t *p, int64_t values) {
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < values; i += static_cast<int64_t>(gridDim.x) * 256) p[i] = 0;
}

// Workspace of the forward: x and weight quantised, and the product's own
struct ForwardLayout {
    int64_t ld, bk, bm;
    size_t off_x, off_sx, off_w, off_sw, off_part, bytes;
};
ForwardLayout forward_layout(int64_t n, int64_t K, int64_t M) {
    ForwardLayout L;
    L.ld = round_up(K, 16);
    L.bk = ceil_div(K, kBlock);
    L.bm = ceil_div(M, kBlock);
    size_t o = 0;
    L.off_x = o;     o += align256(static_cast<size_t>(n) * L.ld);
    L.off_sx = o;    o += align256(static_cast<size_t>(n) * L.bk);
    L.off_w = o;     o += align256(static_cast<size_t>(M) * L.ld);
    L.off_sw = o;    o += align256(static_cast<size_t>(L.bm) * L.bk);
    L.off_part = o;
    o += align256(linear_blocks_workspace_bytes(n, K, M));
    L.bytes = o;
    return L;
}

// Workspace of the backward: the two quantised forms of grad_out with their scales, the bias's partial
// sums, and the products' own
struct GradLayout {
    int64_t ldg, ldgt, bm, bn;   // row strides of the 8-bit forms; blocks of M and of n
    size_t off_g, off_gt, off_sg, off_sgt, off_bias, off_part, bytes;
};
GradLayout grad_layout(int64_t n, int64_t K, int64_t M) {
    GradLayout L;
    L.ldg = round_up(M, 16);
    L.ldgt = round_up(n, 16);
    L.bm = ceil_div(M, kBlock);
    L.bn = ceil_div(n, kBlock);
    size_t o = 0;
    L.off_g = o;     o += align256(static_cast<size_t>(n) * L.ldg);
    L.off_gt = o;    o += align256(static_cast<size_t>(M) * L.ldgt);
    L.off_sg = o;    o += align256(static_cast<size_t>(n) * L.bm);
    L.off_sgt = o;   o += align256(static_cast<size_t>(M) * L.bn);
    L.off_bias = o;  o += align256(static_cast<size_t>(L.bn) * M * 4);
    L.off_part = o;
    o += align256(std::max(linear_blocks_workspace_bytes(n, M, K), linear_blocks_workspace_bytes(M, n, K)));
    L.bytes = o;
    return L;
}

}  // namespace

size_t linear_blocks_workspace_bytes(int64_t n, int64_t K, int64_t M) {
    if (n <= 0 || M <= 0 || K <= 0) return 0;
    const int splits = std::max(plan_of(n, K, M, true).splits, plan_of(n, K, M, false).splits);   // whatever the scales' type
    return splits > 1 ? static_cast<size_t>(splits) * n * round_up(M, 8) * 4 : 0;
}

hipError_t launch_linear_blocks(const BlocksArgs &a, hipStream_t st) {
    if (a.n <= 0 || a.M <= 0) return hipSuccess;
    const bool pow2 = a.sx.e8m0 && a.sw.e8m0;
    const Plan p = plan_of(a.n, a.K, a.M, pow2);
    const ShapeInfo &s = kShapes[p.shape];
    blocks::Args g;
    g.w = static_cast<const unsigned char *>(a.weight);
    g.x = static_cast<const unsigned char *>(a.x);
    g.ldw = a.ldw;
    g.ldx = a.ldx;
    g.K = static_cast<int>(a.K);
    g.n = static_cast<int>(a.n);
    g.M = static_cast<int>(a.M);
    const int64_t tf = ceil_div(a.M, s.bf), tt = ceil_div(a.n, s.bt), total = tf * tt * p.splits;
    if (round_up(total, 8) * s.threads > kMaxThreads) return hipErrorInvalidValue;   // outputs past the card's memory
    g.tiles_f = static_cast<int>(tf);
    g.tiles_t = static_cast<int>(tt);
    g.splits = p.splits;
    g.per_xcd = static_cast<int>(ceil_div(total, 8));
    g.sx = a.sx;
    g.sw = a.sw;
    g.part = a.part;
    g.ldpart = round_up(a.M, 8);
    linear::Epi &e = g.e;
    e.scale_x = e.scale_w = nullptr;
    e.bias = a.bias;
    e.bias_bf16 = a.bias_bf16;
    e.act = a.act;
    e.residual = a.residual;
    e.ldr = a.ldr;
    e.out = a.out;
    e.ldo = a.ldo;
    e.out_bf16 = true;
    e.streams = false;
    e.preact = a.preact;
    e.ldp = a.ldp;
    e.n = a.n;
    e.M = a.M;
    hipError_t err;
    switch (p.shape) {
        case BIG: err = launch_shape<Big>(g, pow2, st); break;
        case WIDE: err = launch_shape<Wide>(g, pow2, st); break;
        case LOW: err = launch_shape<Low>(g, pow2, st); break;
        case TINY: err = launch_shape<Tiny>(g, pow2, st); break;
        case ROWS16: err = launch_rows<1>(g, pow2, st); break;
        default: err = launch_rows<2>(g, pow2, st); break;
    }
    if (err != hipSuccess || p.splits == 1) return err;
    const int64_t items = a.n * (g.ldpart / 8);
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(ceil_div(items, 256), 16384))), block(256);
    static_assert(kMaxSplits <= 16, "the fold's loads");
    if (p.splits <= 4) hipLaunchKernelGGL((blocks::blocks_fold_kernel<4>), grid, block, 0, st, a.part, g.ldpart, p.splits, e);
    else hipLaunchKernelGGL((blocks::blocks_fold_kernel<16>), grid, block, 0, st, a.part, g.ldpart, p.splits, e);
    return hipGetLastError();
}

size_t linear_blocks_forward_workspace_bytes(int64_t n, int64_t K, int64_t M) { return forward_layout(n, K, M).bytes; }

hipError_t launch_linear_blocks_forward(const BlocksForwardArgs &a, hipStream_t st) {
    const ForwardLayout L = forward_layout(a.n, a.K, a.M);
    char *ws = static_cast<char *>(a.workspace);
    auto bytes = [&](size_t off) { return reinterpret_cast<unsigned char *>(ws + off); };
    const int64_t bn = ceil_div(a.n, kBlock);
    QuantizeArgs x{}, w{};
    x.x = a.x;
    x.ldx = a.ldx;
    x.n = a.n;
    x.K = a.K;
    x.q = {bytes(L.off_x), L.ld, ws + L.off_sx, 1, a.n, false, true};
    if (a.xt) x.qt = {static_cast<unsigned char *>(a.xt), a.ldxt, a.scale_xt, bn, 1, true, true};
    w.x = a.weight;
    w.ldx = a.ldw;
    w.n = a.M;
    w.K = a.K;
    w.q = {bytes(L.off_w), L.ld, ws + L.off_sw, L.bk, 1, true, true};
    if (a.wt) w.qt = {static_cast<unsigned char *>(a.wt), a.ldwt, a.scale_wt, L.bm, 1, true, true};
    hipError_t e = launch_quantize_pair(x, w, st);
    if (e != hipSuccess || a.n == 0) return e;
    BlocksArgs g{};
    g.x = ws + L.off_x;
    g.weight = ws + L.off_w;
    g.ldx = g.ldw = L.ld;
    g.n = a.n;
    g.K = a.K;
    g.M = a.M;
    g.sx = {ws + L.off_sx, 1, a.n, true};
    g.sw = {ws + L.off_sw, L.bk, 1, true};
    g.bias = a.bias;
    g.bias_bf16 = a.bias_bf16;
    g.residual = a.residual;
    g.ldr = a.ldr;
    g.out = a.out;
    g.ldo = a.ldo;
    g.part = reinterpret_cast<float *>(ws + L.off_part);
    return launch_linear_blocks(g, st);
}

size_t linear_blocks_backward_workspace_bytes(int64_t n, int64_t K, int64_t M) { return grad_layout(n, K, M).bytes; }

hipError_t launch_linear_blocks_backward(const BlocksGradArgs &a, hipStream_t st) {
    const GradLayout L = grad_layout(a.n, a.K, a.M);
    char *ws = static_cast<char *>(a.workspace);
    float *bias_part = reinterpret_cast<float *>(ws + L.off_bias);
    hipError_t e;
    if (a.n > 0) {
        QuantizeArgs q{};
        q.x = a.grad_out;
        q.ldx = a.ldg;
        q.n = a.n;
        q.K = a.M;
        if (a.grad_x) q.q = {reinterpret_cast<unsigned char *>(ws + L.off_g), L.ldg, ws + L.off_sg, 1, a.n, false, true};
        if (a.grad_weight) q.qt = {reinterpret_cast<unsigned char *>(ws + L.off_gt), L.ldgt, ws + L.off_sgt, 1, a.M, false, true};
        q.part = a.grad_bias ? bias_part : nullptr;
        if (a.grad_x || a.grad_weight || a.grad_bias)
            if ((e = launch_quantize_blocks(q, a.grad_bf16, st)) != hipSuccess) return e;
    }
    if (a.grad_bias && (e = launch_column_fold(bias_part, L.bn, a.M, a.M, a.grad_bias, a.grad_bias_bf16, st)) != hipSuccess)
        return e;
    if (a.grad_x && a.n > 0) {
        BlocksArgs g{};
        g.x = ws + L.off_g;
        g.ldx = L.ldg;
        g.sx = {ws + L.off_sg, 1, a.n, true};
        g.weight = a.wt;
        g.ldw = a.ldwt;
        g.sw = a.swt;
        g.n = a.n;
        g.K = a.M;
        g.M = a.K;
        g.out = a.grad_x;
        g.ldo = a.ldgx;
        g.part = reinterpret_cast<float *>(ws + L.off_part);
        if ((e = launch_linear_blocks(g, st)) != hipSuccess) return e;
    }
    if (a.grad_weight && a.n == 0) {
        const int64_t values = a.M * a.K;
        hipLaunchKernelGGL(zero_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(ceil_div(values, 256), 16384))), dim3(256), 0,
                           st, static_cast<uint16_t *>(a.grad_weight), values);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    } else if (a.grad_weight) {
        BlocksArgs g{};
        g.x = ws + L.off_gt;
        g.ldx = L.ldgt;
        g.sx = {ws + L.off_sgt, 1, a.M, true};
        g.weight = a.xt;
        g.ldw = a.ldxt;
        g.sw = a.sxt;
        g.n = a.M;
        g.K = a.n;
        g.M = a.K;
        g.out = a.grad_weight;
        g.ldo = a.K;
        g.part = reinterpret_cast<float *>(ws + L.off_part);
        if ((e = launch_linear_blocks(g, st)) != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace lce
