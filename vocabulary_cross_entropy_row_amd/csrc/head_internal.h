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

}  // namespace lce
