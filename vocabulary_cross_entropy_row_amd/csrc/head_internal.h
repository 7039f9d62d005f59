// Internal interface between the C-ABI host layer (lce_api.cpp) and the kernels
// of the operators around the cross-entropy: the final norm, the rules on its
// logits and the head's matrix product.  Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lce {

// ---- root-mean-square norm ----------------------------------------------------

// Widest row the norm holds in registers: 1024 threads x 16 values.
constexpr int64_t kNormMaxH = 16384;
// Most partial rows of the weight's gradient (one per workgroup of the backward).
constexpr int64_t kNormMaxGroups = 1024;

struct NormArgs {
    const void *x;         // [n, H], row stride ldx
    const void *residual;  // [n, H], row stride ldr, or NULL
    const void *weight;    // [H] or NULL (ones)
    void *sum;             // [n, H], row stride lds, or NULL
    void *y;               // [n, H], row stride ldy: x's type, or e4m3
    float *rstd;           // [n] or NULL
    float *scale;          // [n] (e4m3 only)
    int64_t ldx, ldr, lds, ldy, n, H;
    float eps, offset;     // offset: added to the weight
    bool weight_bf16, out8;
    int64_t row0 = 0;      // first row of a launch
};
hipError_t launch_rms_norm(const NormArgs &a, bool is_bf16, hipStream_t st);

struct NormGradArgs {
    const void *gy;        // [n, H], row stride ldg
    const void *s;         // the normalised rows (x, or x + residual), row stride lds
    const void *weight;    // [H] or NULL
    const void *gs;        // upstream gradient of the sum, row stride ldgs, or NULL
    const float *rstd;     // [n]
    void *gx;              // [n, H], row stride ldgx
    void *gw;              // [H] fp32 or bf16, or NULL
    float *part;           // [norm_groups][H]
    int64_t ldg, lds, ldgs, ldgx, n, H;
    float offset;
    bool weight_bf16, gw_bf16;
};
hipError_t launch_rms_norm_backward(const NormGradArgs &a, bool is_bf16, hipStream_t st);

// out[c] = sum over rows of part[row][c] (row stride ld), in row order within
// eight interleaved groups: the same order every time.
hipError_t launch_column_fold(const float *part, int64_t rows, int64_t ld, int64_t cols, void *out, bool out_bf16,
                              hipStream_t st);

// ---- rules on logits ------------------------------------------------------------

struct RulesArgs {
    const void *logits;        // [n, V], row stride ldx
    void *out;                 // [n, V], row stride ldo (may be the logits)
    int64_t ldx, ldo, n, V;
    const void *history;       // [n, L] token ids, row stride ldh, or NULL
    int64_t ldh, L;
    const int64_t *history_lens, *prompt_lens;   // [n] or NULL
    const void *bias_ids;      // [n, B] token ids, row stride ldbi, or NULL
    const float *bias_values;  // [n, B], row stride ldbv
    int64_t ldbi, ldbv, B;
    bool id64;                 // ids are int64, else int32
    const float *repetition, *presence, *frequency, *temperature;   // [n] or NULL
    const uint32_t *allowed;   // [R, ceil(V / 32)] bits, row stride ldm words, or NULL
    int64_t ldm, R;
    const int64_t *mask_rows;  // [n] or NULL (row i uses mask row i)
    float mask_value, softcap;
};
hipError_t launch_logits_process(const RulesArgs &a, bool is_bf16, hipStream_t st);

// ---- matrix product with an epilogue ----------------------------------------------

// Longest row stride of what the product reads, in bytes: 256 rows, the most of a tile, and one step of
// K read ahead keep 32-bit offsets.
constexpr int64_t kLinearMaxStride = (int64_t(1) << 32) / 256 - 1024;

enum Act { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

struct LinearArgs {
    const void *x;         // [n, K] bf16 or e4m3, row stride ldx (elements)
    const void *weight;    // [M, K] of the same type, row stride ldw
    int64_t ldx, ldw, n, K, M;
    bool fp8;
    const float *scale_x;  // [n] or NULL
    const float *scale_w;  // [M] or NULL
    const void *bias;      // [M] or NULL
    bool bias_bf16;
    int act;
    const void *residual;  // [n, M] of the output's type, row stride ldr, or NULL
    int64_t ldr;
    void *out;             // [n, M] bf16 or fp32, row stride ldo
    int64_t ldo;
    bool out_bf16;
    void *preact;          // [n, M] bf16, row stride ldp, or NULL
    int64_t ldp;
    float *part;           // workspace: split partials [splits][n][round8(M)] fp32
};
// Bytes of split partials the product needs (0: it is not split).
size_t linear_workspace_bytes(int64_t n, int64_t K, int64_t M, bool fp8);
hipError_t launch_linear(const LinearArgs &a, hipStream_t st);

struct LinearGradArgs {
    const void *grad_out;  // [n, M] bf16 or fp32, row stride ldg
    int64_t ldg;
    bool grad_bf16;
    const void *x;         // [n, K] bf16, row stride ldx
    const void *weight;    // [M, K] bf16, row stride ldw
    int64_t ldx, ldw;
    const void *preact;    // [n, M] bf16, row stride ldp (act other than none)
    int64_t ldp;
    int act;
    int64_t n, K, M;
    void *grad_x;          // [n, K] bf16, row stride ldgx, or NULL
    int64_t ldgx;
    void *grad_weight;     // [M, K] bf16 or fp32, contiguous, or NULL
    bool grad_weight_bf16;
    void *grad_bias;       // [M] bf16 or fp32, or NULL
    bool grad_bias_bf16;
    void *workspace;
};
size_t linear_backward_workspace_bytes(int64_t n, int64_t K, int64_t M);
hipError_t launch_linear_backward(const LinearGradArgs &a, hipStream_t st);

}  // namespace lce
