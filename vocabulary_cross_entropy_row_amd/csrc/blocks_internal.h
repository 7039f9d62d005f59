// Internal interface between the C-ABI host layer (lce_api.cpp) and the kernels of the 8-bit products
// with a scale for each block of 128 and of the orthogonalised update.  Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lce {

constexpr int64_t kBlock = 128;   // values of K (and, in tiles, rows) that share a scale

// ---- quantiser ---------------------------------------------------------------------

// One quantised matrix: values [rows, cols] e4m3, row stride ld; scales [rows or ceil(rows / 128),
// ceil(cols / 128)] with strides s_row, s_col (elements).
struct BlockedOut {
    unsigned char *values;   // NULL: not wanted
    int64_t ld;
    void *scale;
    int64_t s_row, s_col;
    bool tile;               // blocks of 128 x 128, not 1 x 128
    bool e8m0;               // scales as exponents in a byte, else fp32
};
struct QuantizeArgs {
    const void *x;           // [n, K] row stride ldx
    int64_t ldx, n, K;
    BlockedOut q, qt;        // of x and of its transpose
    float *part;             // column sums of each 128 rows, [ceil(n / 128)][K], or NULL
};
hipError_t launch_quantize_blocks(const QuantizeArgs &a, bool is_bf16, hipStream_t st);
// Two bf16 matrices in one launch
hipError_t launch_quantize_pair(const QuantizeArgs &a, const QuantizeArgs &b, hipStream_t st);

// ---- product -------------------------------------------------------------------------

struct Scales {
    const void *p;
    int64_t s_row, s_col;    // elements, per row of the operand (x) or 128 rows (weight), and per block of K
    bool e8m0;
};
struct BlocksArgs {
    const void *x, *weight;  // e4m3 [n, K], [M, K]
    int64_t ldx, ldw, n, K, M;
    Scales sx, sw;
    const void *bias;        // [M] or NULL
    bool bias_bf16;
    int act;
    const void *residual;    // [n, M] bf16, row stride ldr, or NULL
    int64_t ldr;
    void *out;               // [n, M] bf16, row stride ldo
    int64_t ldo;
    void *preact;            // [n, M] bf16, row stride ldp, or NULL
    int64_t ldp;
    float *part;             // workspace
};
size_t linear_blocks_workspace_bytes(int64_t n, int64_t K, int64_t M);
hipError_t launch_linear_blocks(const BlocksArgs &a, hipStream_t st);

struct BlocksForwardArgs {
    const void *x, *weight;  // bf16 [n, K], [M, K]
    int64_t ldx, ldw, n, K, M;
    const void *bias;        // [M] or NULL
    bool bias_bf16;
    const void *residual;    // [n, M] bf16, row stride ldr, or NULL
    int64_t ldr;
    void *out;               // [n, M] bf16, row stride ldo
    int64_t ldo;
    void *xt, *wt;           // e4m3 [K, n] and [K, M] in tiles, for the backward, or NULL
    int64_t ldxt, ldwt;
    void *scale_xt, *scale_wt;   // e8m0, contiguous
    void *workspace;
};
size_t linear_blocks_forward_workspace_bytes(int64_t n, int64_t K, int64_t M);
hipError_t launch_linear_blocks_forward(const BlocksForwardArgs &a, hipStream_t st);

struct BlocksGradArgs {
    const void *grad_out;    // [n, M] bf16 or fp32, row stride ldg
    int64_t ldg;
    bool grad_bf16;
    const void *xt;          // x transposed, e4m3 [K, n], tiles
    int64_t ldxt;
    Scales sxt;
    const void *wt;          // weight transposed, e4m3 [K, M], tiles
    int64_t ldwt;
    Scales swt;
    int64_t n, K, M;
    void *grad_x;            // [n, K] bf16, row stride ldgx, or NULL
    int64_t ldgx;
    void *grad_weight;       // [M, K] bf16, contiguous, or NULL
    void *grad_bias;         // [M] or NULL
    bool grad_bias_bf16;
    void *workspace;
};
size_t linear_blocks_backward_workspace_bytes(int64_t n, int64_t K, int64_t M);
hipError_t launch_linear_blocks_backward(const BlocksGradArgs &a, hipStream_t st);

// ---- orthogonalised update -------------------------------------------------------------

struct OrthoArgs {
    const void *g;           // [batch][rows, cols], strides in elements
    int64_t ldg, batch_stride, batch, rows, cols;
    bool g_bf16;
    void *out;               // bf16, the same shape
    int64_t ldo, out_batch_stride;
    int steps;
    float a, b, c, eps;
    void *workspace;
};
size_t orthogonalise_workspace_bytes(int64_t batch, int64_t rows, int64_t cols);
hipError_t launch_orthogonalise(const OrthoArgs &a, hipStream_t st);

}  // namespace lce
