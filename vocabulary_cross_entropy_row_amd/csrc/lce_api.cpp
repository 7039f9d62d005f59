// C-ABI entry points (include/lce.h): argument validation, then kernel launch.
// Validation runs before any HIP call, so every argument error is reported
// without touching the device.  No exception crosses the ABI.
#include "lce.h"

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <atomic>
#include <mutex>

#include "blocks_internal.h"
#include "head_internal.h"
#include "lce_internal.h"
#include "ortho_plan.h"

// The workspace of lce_ce_fwd_bwd_noalloc: room for the row kernel's workspace
// at any n (its per-workgroup part stops growing at kMaxRowGroups workgroups),
// one copy per device, held until the process ends.  Host code never uses this
// name as an address: it is a host-side stand-in for the device symbol, whose
// address on each device comes from hipGetSymbolAddress (noalloc_scratch).
constexpr size_t kNoAllocScratchBytes = lce::ce_workspace_bytes(lce::kMaxRowGroups);
static __device__ __align__(256) unsigned char scratch[kNoAllocScratchBytes];

namespace {

thread_local char g_err[512] = "";

lce_status fail(lce_status st, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return st;
}

lce_status ok() {
    g_err[0] = '\0';
    return LCE_OK;
}

lce_status hip_status(hipError_t e, const char *what) {
    if (e == hipSuccess) return ok();
    return fail(LCE_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool is_aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Checks shared by the tile-resident fused linear entry points.
lce_status check_flce_resident(const char *fn, const void *hidden, const void *weight, const int64_t *labels,
                               int64_t n, int64_t H, int64_t V, float label_smoothing, float softcap,
                               lce_reduction reduction) {
    if (n < 0) return fail(LCE_ERR_INVALID_ARG, "%s: n must be >= 0 (got %lld)", fn, (long long)n);
    if (H < 1) return fail(LCE_ERR_INVALID_ARG, "%s: H must be >= 1 (got %lld)", fn, (long long)H);
    if (V < 1) return fail(LCE_ERR_INVALID_ARG, "%s: V must be >= 1 (got %lld)", fn, (long long)V);
    if (reduction != LCE_RED_NONE && reduction != LCE_RED_MEAN && reduction != LCE_RED_SUM)
        return fail(LCE_ERR_INVALID_ARG, "%s: unknown reduction %d", fn, (int)reduction);
    if (!(label_smoothing >= 0.0f && label_smoothing <= 1.0f))
        return fail(LCE_ERR_INVALID_ARG, "%s: label_smoothing must be in [0, 1] (got %g)", fn, (double)label_smoothing);
    if (!(softcap >= 0.0f) || isinf(softcap))
        return fail(LCE_ERR_INVALID_ARG, "%s: softcap must be finite and >= 0 (got %g)", fn, (double)softcap);
    if (!weight) return fail(LCE_ERR_INVALID_ARG, "%s: weight is required", fn);
    if (n > 0 && (!hidden || !labels)) return fail(LCE_ERR_INVALID_ARG, "%s: hidden and labels are required", fn);
    if (H % 8 != 0 || V % 8 != 0)
        return fail(LCE_ERR_UNSUPPORTED, "%s: requires H and V to be multiples of 8 (16-byte bf16 rows); got H=%lld V=%lld",
                    fn, (long long)H, (long long)V);
    if ((hidden && !is_aligned(hidden, 16)) || !is_aligned(weight, 16))
        return fail(LCE_ERR_UNSUPPORTED, "%s: hidden and weight must be 16-byte aligned", fn);
    if (n > 0x7fffffffLL || V > 0x7fffffffLL / 16 || H > 0x7fffffffLL / 16 || 256ull * V * 2 >= (1ull << 32) ||
        256ull * H * 2 >= (1ull << 32))
        return fail(LCE_ERR_UNSUPPORTED, "%s: n >= 2^31 or a 256-row operand tile exceeds 4 GiB", fn);
    return LCE_OK;
}

}  // namespace

extern "C" {

int lce_abi_version(void) { return 3; }

const char *lce_last_error(void) { return g_err; }

size_t lce_ce_workspace_bytes(int64_t n, int64_t V) {
    (void)V;
    return lce::ce_workspace_bytes(n);
}

}  // extern "C"

namespace {

// Checks of lce_ce_fwd_bwd's arguments other than the workspace, in the order the
// header lists them; the call's name prefixes every message.
lce_status check_ce_args(const char *fn, const void *logits_inout, int64_t ld, lce_dtype dtype,
                         const int64_t *labels, int64_t n, int64_t V, float label_smoothing, float softcap,
                         lce_reduction reduction, const float *loss_tok, const int64_t *counts) {
    if (n < 0) return fail(LCE_ERR_INVALID_ARG, "%s: n must be >= 0 (got %lld)", fn, (long long)n);
    if (V < 1) return fail(LCE_ERR_INVALID_ARG, "%s: V must be >= 1 (got %lld)", fn, (long long)V);
    if (ld < V) return fail(LCE_ERR_INVALID_ARG, "%s: ld (%lld) must be >= V (%lld)", fn, (long long)ld, (long long)V);
    if (dtype != LCE_F32 && dtype != LCE_BF16) return fail(LCE_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    if (reduction != LCE_RED_NONE && reduction != LCE_RED_MEAN && reduction != LCE_RED_SUM)
        return fail(LCE_ERR_INVALID_ARG, "%s: unknown reduction %d", fn, (int)reduction);
    if (!(label_smoothing >= 0.0f && label_smoothing <= 1.0f))
        return fail(LCE_ERR_INVALID_ARG, "%s: label_smoothing must be in [0, 1] (got %g)", fn, (double)label_smoothing);
    if (!(softcap >= 0.0f) || isinf(softcap))
        return fail(LCE_ERR_INVALID_ARG, "%s: softcap must be finite and >= 0 (got %g)", fn, (double)softcap);
    if (!counts) return fail(LCE_ERR_INVALID_ARG, "%s: counts is required", fn);
    if (n > 0) {
        if (!logits_inout) return fail(LCE_ERR_INVALID_ARG, "%s: logits is required", fn);
        if (!labels) return fail(LCE_ERR_INVALID_ARG, "%s: labels is required", fn);
        if (!loss_tok) return fail(LCE_ERR_INVALID_ARG, "%s: loss_tok is required", fn);
        const size_t esz = dtype == LCE_BF16 ? 2 : 4;
        if (!is_aligned(logits_inout, esz))
            return fail(LCE_ERR_INVALID_ARG, "%s: logits must be aligned to its element size", fn);
    }
    return LCE_OK;
}

lce_status launch_ce(const char *fn, void *logits_inout, int64_t ld, lce_dtype dtype, const int64_t *labels, int64_t n,
                     int64_t V, int64_t ignore_index, float label_smoothing, float softcap, lce_reduction reduction,
                     const float *grad_out, float *loss_tok, float *loss_out, int64_t *argmax_out, int64_t *counts,
                     void *workspace, hipStream_t stream) {
    if (n > 0x7fffffffLL) return fail(LCE_ERR_UNSUPPORTED, "%s: n > 2^31-1 rows is not supported", fn);
    if (V > 0x7fffffffLL / 16) return fail(LCE_ERR_UNSUPPORTED, "%s: V > 2^27 columns is not supported", fn);
    lce::CEArgs a;
    a.logits = logits_inout;
    a.ld = ld;
    a.n = n;
    a.V = V;
    a.labels = labels;
    a.count_labels = labels;
    a.count_n = n;
    a.ignore_index = ignore_index;
    a.eps = label_smoothing;
    a.softcap = softcap;
    a.reduction = static_cast<int>(reduction);
    a.grad_out = grad_out;
    a.loss_tok = loss_tok;
    a.loss_out = loss_out;
    a.argmax_out = argmax_out;
    a.counts = counts;
    a.workspace = workspace;
    char what[64];
    snprintf(what, sizeof what, "%s launch", fn);
    return hip_status(lce::launch_ce_fwd_bwd(a, dtype == LCE_BF16, stream), what);
}

// Device address of `scratch` on each device, looked up by the first
// lce_ce_fwd_bwd_noalloc call on that device (with the device current).
constexpr int kMaxDevices = 64;
std::atomic<void *> g_scratch[kMaxDevices];
std::mutex g_scratch_mu;   // taken only until a device's address is known

lce_status noalloc_scratch(const char *fn, hipStream_t stream, void **out) {
    int dev = -1;
    hipError_t e = hipStreamGetDevice(stream, &dev);
    if (e != hipSuccess) return hip_status(e, "lce_ce_fwd_bwd_noalloc: hipStreamGetDevice");
    if (dev < 0 || dev >= kMaxDevices)
        return fail(LCE_ERR_UNSUPPORTED, "%s: device %d is beyond the %d devices the scratch table holds", fn, dev,
                    kMaxDevices);
    void *p = g_scratch[dev].load(std::memory_order_acquire);
    if (!p) {
        std::lock_guard<std::mutex> lock(g_scratch_mu);
        p = g_scratch[dev].load(std::memory_order_acquire);
        if (!p) {
            int cur = -1;
            if ((e = hipGetDevice(&cur)) != hipSuccess) return hip_status(e, "lce_ce_fwd_bwd_noalloc: hipGetDevice");
            if (cur != dev && (e = hipSetDevice(dev)) != hipSuccess)
                return hip_status(e, "lce_ce_fwd_bwd_noalloc: hipSetDevice");
            e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
            const hipError_t back = cur != dev ? hipSetDevice(cur) : hipSuccess;
            if (e != hipSuccess) return hip_status(e, "lce_ce_fwd_bwd_noalloc: hipGetSymbolAddress");
            if (back != hipSuccess) return hip_status(back, "lce_ce_fwd_bwd_noalloc: hipSetDevice");
            if (!p) return fail(LCE_ERR_HIP, "%s: hipGetSymbolAddress gave a null address", fn);
            g_scratch[dev].store(p, std::memory_order_release);
        }
    }
    *out = p;
    return LCE_OK;
}

}  // namespace

extern "C" {

lce_status lce_ce_fwd_bwd(void *logits_inout, int64_t ld, lce_dtype dtype, const int64_t *labels, int64_t n,
                          int64_t V, int64_t ignore_index, float label_smoothing, float softcap,
                          lce_reduction reduction, const float *grad_out, float *loss_tok, float *loss_out,
                          int64_t *argmax_out, int64_t *counts, void *workspace, size_t workspace_bytes,
                          hipStream_t stream) {
    const char *fn = "lce_ce_fwd_bwd";
    lce_status st = check_ce_args(fn, logits_inout, ld, dtype, labels, n, V, label_smoothing, softcap, reduction,
                                  loss_tok, counts);
    if (st != LCE_OK) return st;
    if (!workspace) return fail(LCE_ERR_INVALID_ARG, "%s: workspace is required", fn);
    if (workspace_bytes < lce_ce_workspace_bytes(n, V))
        return fail(LCE_ERR_INVALID_ARG, "%s: workspace_bytes %zu < required %zu", fn, workspace_bytes,
                    lce_ce_workspace_bytes(n, V));
    if (!is_aligned(workspace, 16)) return fail(LCE_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", fn);
    return launch_ce(fn, logits_inout, ld, dtype, labels, n, V, ignore_index, label_smoothing, softcap, reduction,
                     grad_out, loss_tok, loss_out, argmax_out, counts, workspace, stream);
}

lce_status lce_ce_fwd_bwd_noalloc(void *logits_inout, int64_t ld, lce_dtype dtype, const int64_t *labels, int64_t n,
                                  int64_t V, int64_t ignore_index, float label_smoothing, float softcap,
                                  lce_reduction reduction, const float *grad_out, float *loss_tok, float *loss_out,
                                  int64_t *argmax_out, int64_t *counts, hipStream_t stream) {
    const char *fn = "lce_ce_fwd_bwd_noalloc";
    lce_status st = check_ce_args(fn, logits_inout, ld, dtype, labels, n, V, label_smoothing, softcap, reduction,
                                  loss_tok, counts);
    if (st != LCE_OK) return st;
    if (lce_ce_workspace_bytes(n, V) > kNoAllocScratchBytes)
        return fail(LCE_ERR_UNSUPPORTED, "%s: needs %zu bytes of scratch, more than the %zu it holds", fn,
                    lce_ce_workspace_bytes(n, V), kNoAllocScratchBytes);
    void *ws = nullptr;
    if ((st = noalloc_scratch(fn, stream, &ws)) != LCE_OK) return st;
    return launch_ce(fn, logits_inout, ld, dtype, labels, n, V, ignore_index, label_smoothing, softcap, reduction,
                     grad_out, loss_tok, loss_out, argmax_out, counts, ws, stream);
}

lce_status lce_ce_argmax(const void *logits, int64_t ld, lce_dtype dtype, const int64_t *labels, int64_t n,
                         int64_t V, int64_t ignore_index, int64_t *argmax_out, int64_t *counts,
                         hipStream_t stream) {
    if (n < 0) return fail(LCE_ERR_INVALID_ARG, "lce_ce_argmax: n must be >= 0 (got %lld)", (long long)n);
    if (V < 1) return fail(LCE_ERR_INVALID_ARG, "lce_ce_argmax: V must be >= 1 (got %lld)", (long long)V);
    if (ld < V) return fail(LCE_ERR_INVALID_ARG, "lce_ce_argmax: ld (%lld) must be >= V (%lld)", (long long)ld,
                            (long long)V);
    if (dtype != LCE_F32 && dtype != LCE_BF16)
        return fail(LCE_ERR_INVALID_ARG, "lce_ce_argmax: unknown dtype %d", (int)dtype);
    if (!counts) return fail(LCE_ERR_INVALID_ARG, "lce_ce_argmax: counts is required");
    if (n > 0) {
        if (!logits) return fail(LCE_ERR_INVALID_ARG, "lce_ce_argmax: logits is required");
        if (!argmax_out) return fail(LCE_ERR_INVALID_ARG, "lce_ce_argmax: argmax_out is required");
        const size_t esz = dtype == LCE_BF16 ? 2 : 4;
        if (!is_aligned(logits, esz))
            return fail(LCE_ERR_INVALID_ARG, "lce_ce_argmax: logits must be aligned to its element size");
    }
    if (n > 0x7fffffffLL) return fail(LCE_ERR_UNSUPPORTED, "lce_ce_argmax: n > 2^31-1 rows is not supported");
    if (V > 0x7fffffffLL / 16) return fail(LCE_ERR_UNSUPPORTED, "lce_ce_argmax: V > 2^27 columns is not supported");
    return hip_status(lce::launch_ce_argmax(logits, ld, dtype == LCE_BF16, labels, n, V, ignore_index, argmax_out,
                                            counts, stream),
                      "lce_ce_argmax launch");
}

// shared checks of a logits shard [n, Vs] with row stride ld
static lce_status check_shard(const char *fn, const void *logits, int64_t ld, lce_dtype dtype, const int64_t *labels,
                              int64_t n, int64_t Vs, int64_t v0) {
    if (n < 0) return fail(LCE_ERR_INVALID_ARG, "%s: n must be >= 0 (got %lld)", fn, (long long)n);
    if (Vs < 1) return fail(LCE_ERR_INVALID_ARG, "%s: the shard width must be >= 1 (got %lld)", fn, (long long)Vs);
    if (v0 < 0) return fail(LCE_ERR_INVALID_ARG, "%s: v_offset must be >= 0 (got %lld)", fn, (long long)v0);
    if (ld < Vs) return fail(LCE_ERR_INVALID_ARG, "%s: ld (%lld) must be >= the shard width (%lld)", fn,
                             (long long)ld, (long long)Vs);
    if (dtype != LCE_F32 && dtype != LCE_BF16) return fail(LCE_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    if (n > 0 && (!logits || !labels)) return fail(LCE_ERR_INVALID_ARG, "%s: logits and labels are required", fn);
    const int64_t E = dtype == LCE_BF16 ? 8 : 4;
    if (Vs % E != 0 || ld % E != 0 || (logits && !is_aligned(logits, 16)))
        return fail(LCE_ERR_UNSUPPORTED,
                    "%s: requires 16-byte rows (shard width and ld multiples of %lld elements, 16-byte aligned logits)",
                    fn, (long long)E);
    if (n > 0x7fffffffLL) return fail(LCE_ERR_UNSUPPORTED, "%s: n > 2^31-1 rows is not supported", fn);
    if (v0 + Vs > 0x7fffffffLL || Vs * (dtype == LCE_BF16 ? 2 : 4) >= (1ll << 32))
        return fail(LCE_ERR_UNSUPPORTED, "%s: vocabulary indexes must fit 31 bits and a shard row 4 GiB", fn);
    return LCE_OK;
}

size_t lce_ce_stats_bytes(int64_t n) { return n < 0 ? 0 : static_cast<size_t>(n) * lce::kStatsFloats * sizeof(float); }

lce_status lce_ce_stats(const void *logits, int64_t ld, lce_dtype dtype, const int64_t *labels, int64_t n,
                        int64_t shard_V, int64_t v_offset, int64_t ignore_index, float softcap, float *stats,
                        hipStream_t stream) {
    const char *fn = "lce_ce_stats";
    lce_status st = check_shard(fn, logits, ld, dtype, labels, n, shard_V, v_offset);
    if (st != LCE_OK) return st;
    if (!(softcap >= 0.0f) || isinf(softcap))
        return fail(LCE_ERR_INVALID_ARG, "%s: softcap must be finite and >= 0 (got %g)", fn, (double)softcap);
    if (n > 0 && !stats) return fail(LCE_ERR_INVALID_ARG, "%s: stats is required", fn);
    return hip_status(lce::launch_ce_stats(logits, ld, dtype == LCE_BF16, labels, n, shard_V, v_offset, ignore_index,
                                           softcap, stats, stream),
                      "lce_ce_stats launch");
}

lce_status lce_ce_combine(const float *stats, int64_t shards, const int64_t *labels, int64_t n, int64_t V,
                          int64_t ignore_index, float label_smoothing, lce_reduction reduction, float *lse,
                          float *one_minus_py, float *loss_tok, float *loss_out, float *logprob, float *entropy,
                          int64_t *argmax_out, int64_t *counts, hipStream_t stream) {
    const char *fn = "lce_ce_combine";
    if (n < 0) return fail(LCE_ERR_INVALID_ARG, "%s: n must be >= 0 (got %lld)", fn, (long long)n);
    if (V < 1) return fail(LCE_ERR_INVALID_ARG, "%s: V must be >= 1 (got %lld)", fn, (long long)V);
    if (shards < 1) return fail(LCE_ERR_INVALID_ARG, "%s: shards must be >= 1 (got %lld)", fn, (long long)shards);
    if (reduction != LCE_RED_NONE && reduction != LCE_RED_MEAN && reduction != LCE_RED_SUM)
        return fail(LCE_ERR_INVALID_ARG, "%s: unknown reduction %d", fn, (int)reduction);
    if (!(label_smoothing >= 0.0f && label_smoothing <= 1.0f))
        return fail(LCE_ERR_INVALID_ARG, "%s: label_smoothing must be in [0, 1] (got %g)", fn, (double)label_smoothing);
    if (!counts) return fail(LCE_ERR_INVALID_ARG, "%s: counts is required", fn);
    if (n > 0 && (!stats || !labels || !lse))
        return fail(LCE_ERR_INVALID_ARG, "%s: stats, labels and lse are required", fn);
    if (n > 0 && loss_out && !loss_tok) return fail(LCE_ERR_INVALID_ARG, "%s: loss_out needs loss_tok", fn);
    if (n > 0x7fffffffLL) return fail(LCE_ERR_UNSUPPORTED, "%s: n > 2^31-1 rows is not supported", fn);
    return hip_status(lce::launch_ce_combine(stats, shards, n, 1, labels, n, V, ignore_index, label_smoothing,
                                             static_cast<int>(reduction), lse, one_minus_py, loss_tok, loss_out,
                                             logprob, entropy, argmax_out, counts, stream),
                      "lce_ce_combine launch");
}

lce_status lce_ce_grad(void *logits_inout, int64_t ld, lce_dtype dtype, const int64_t *labels, int64_t n,
                       int64_t shard_V, int64_t v_offset, int64_t V, int64_t ignore_index, float label_smoothing,
                       float softcap, lce_reduction reduction, const float *grad_out, const float *lse,
                       const float *one_minus_py, const int64_t *counts, hipStream_t stream) {
    const char *fn = "lce_ce_grad";
    lce_status st = check_shard(fn, logits_inout, ld, dtype, labels, n, shard_V, v_offset);
    if (st != LCE_OK) return st;
    if (V < 1 || v_offset + shard_V > V)
        return fail(LCE_ERR_INVALID_ARG, "%s: the shard [%lld, %lld) must lie inside [0, V = %lld)", fn,
                    (long long)v_offset, (long long)(v_offset + shard_V), (long long)V);
    if (reduction != LCE_RED_NONE && reduction != LCE_RED_MEAN && reduction != LCE_RED_SUM)
        return fail(LCE_ERR_INVALID_ARG, "%s: unknown reduction %d", fn, (int)reduction);
    if (!(label_smoothing >= 0.0f && label_smoothing <= 1.0f))
        return fail(LCE_ERR_INVALID_ARG, "%s: label_smoothing must be in [0, 1] (got %g)", fn, (double)label_smoothing);
    if (!(softcap >= 0.0f) || isinf(softcap))
        return fail(LCE_ERR_INVALID_ARG, "%s: softcap must be finite and >= 0 (got %g)", fn, (double)softcap);
    if (n > 0 && (!lse || !one_minus_py || !counts))
        return fail(LCE_ERR_INVALID_ARG, "%s: lse, one_minus_py and counts are required", fn);
    return hip_status(lce::launch_ce_grad(logits_inout, ld, dtype == LCE_BF16, labels, n, shard_V, v_offset, V,
                                          ignore_index, label_smoothing, softcap, static_cast<int>(reduction),
                                          grad_out, lse, one_minus_py, counts, stream),
                      "lce_ce_grad launch");
}

size_t lce_flce_workspace_bytes(int64_t n, int64_t H, int64_t V, int64_t chunk_tokens) {
    if (n < 0 || H < 1 || V < 1 || chunk_tokens < 1) return 0;
    return lce::flce_layout(n, H, V, chunk_tokens, lce::flce_default_group_chunks(n, H, V, chunk_tokens), false).bytes;
}

size_t lce_flce_workspace_bytes_grouped(int64_t n, int64_t H, int64_t V, int64_t chunk_tokens, int64_t group_chunks) {
    if (n < 0 || H < 1 || V < 1 || chunk_tokens < 1 || group_chunks < 1) return 0;
    return lce::flce_layout(n, H, V, chunk_tokens, group_chunks, false).bytes;
}

lce_status lce_flce_fwd_bwd(const void *hidden, const void *weight, const int64_t *labels, int64_t n, int64_t H,
                            int64_t V, int64_t ignore_index, float label_smoothing, float softcap,
                            lce_reduction reduction, const float *grad_out, int64_t chunk_tokens, float *loss_tok,
                            float *loss_out, void *grad_hidden, float *grad_weight, int64_t *counts, void *workspace,
                            size_t workspace_bytes, hipStream_t stream, hipStream_t aux_stream) {
    const char *fn = "lce_flce_fwd_bwd";
    if (n < 0) return fail(LCE_ERR_INVALID_ARG, "%s: n must be >= 0 (got %lld)", fn, (long long)n);
    if (H < 1) return fail(LCE_ERR_INVALID_ARG, "%s: H must be >= 1 (got %lld)", fn, (long long)H);
    if (V < 1) return fail(LCE_ERR_INVALID_ARG, "%s: V must be >= 1 (got %lld)", fn, (long long)V);
    if (chunk_tokens < 1) return fail(LCE_ERR_INVALID_ARG, "%s: chunk_tokens must be >= 1", fn);
    if (reduction != LCE_RED_NONE && reduction != LCE_RED_MEAN && reduction != LCE_RED_SUM)
        return fail(LCE_ERR_INVALID_ARG, "%s: unknown reduction %d", fn, (int)reduction);
    if (!(label_smoothing >= 0.0f && label_smoothing <= 1.0f))
        return fail(LCE_ERR_INVALID_ARG, "%s: label_smoothing must be in [0, 1] (got %g)", fn, (double)label_smoothing);
    if (!(softcap >= 0.0f) || isinf(softcap))
        return fail(LCE_ERR_INVALID_ARG, "%s: softcap must be finite and >= 0 (got %g)", fn, (double)softcap);
    if (!weight || !grad_weight || !counts || !workspace)
        return fail(LCE_ERR_INVALID_ARG, "%s: weight, grad_weight, counts and workspace are required", fn);
    if (n > 0 && (!hidden || !labels || !loss_tok || !grad_hidden))
        return fail(LCE_ERR_INVALID_ARG, "%s: hidden, labels, loss_tok and grad_hidden are required", fn);
    // the largest grad_weight group (up to the default) whose layout fits the workspace
    int64_t group = 1;
    bool with_wt = false;
    const bool fits = lce::flce_plan(n, H, V, chunk_tokens, workspace_bytes, &group, &with_wt);
    const size_t need = lce::flce_layout(n, H, V, chunk_tokens, 1, false).bytes;
    if (!fits)
        return fail(LCE_ERR_INVALID_ARG, "%s: workspace_bytes %zu < minimum %zu", fn, workspace_bytes, need);
    if (!is_aligned(workspace, 256)) return fail(LCE_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", fn);
    if (H % 8 != 0 || V % 8 != 0)
        return fail(LCE_ERR_UNSUPPORTED, "%s: requires H and V to be multiples of 8 (16-byte bf16 rows); got H=%lld V=%lld",
                    fn, (long long)H, (long long)V);
    if ((hidden && !is_aligned(hidden, 16)) || !is_aligned(weight, 16) || (grad_hidden && !is_aligned(grad_hidden, 16)) ||
        !is_aligned(grad_weight, 16))
        return fail(LCE_ERR_UNSUPPORTED, "%s: hidden, weight, grad_hidden and grad_weight must be 16-byte aligned", fn);
    const int64_t C = chunk_tokens < n ? chunk_tokens : n;
    if (V > 0x7fffffffLL / 16 || H > 0x7fffffffLL / 16 || C > 0x7fffffffLL / 16 ||
        static_cast<unsigned long long>(C) * V * 2 >= (1ull << 32) || 256ull * V * 2 >= (1ull << 32) ||
        256ull * H * 2 >= (1ull << 32))
        return fail(LCE_ERR_UNSUPPORTED, "%s: a chunk of logits or a 256-row operand tile exceeds 4 GiB", fn);
    if (!with_wt && n > 0 && static_cast<unsigned long long>(V) * H * 2 >= (1ull << 32))
        return fail(LCE_ERR_UNSUPPORTED,
                    "%s: without room for W^T in the workspace the grad_hidden GEMM reads the weight in place, "
                    "which needs V * H * 2 < 4 GiB (V=%lld H=%lld); pass lce_flce_workspace_bytes() bytes", fn,
                    (long long)V, (long long)H);
    lce::FlceArgs f;
    f.hidden = hidden;
    f.weight = weight;
    f.labels = labels;
    f.n = n;
    f.H = H;
    f.V = V;
    f.chunk = chunk_tokens;
    f.ignore_index = ignore_index;
    f.eps = label_smoothing;
    f.softcap = softcap;
    f.reduction = static_cast<int>(reduction);
    f.grad_out = grad_out;
    f.loss_tok = loss_tok;
    f.loss_out = loss_out;
    f.grad_hidden = grad_hidden;
    f.grad_weight = grad_weight;
    f.counts = counts;
    f.workspace = workspace;
    f.group_chunks = group;
    f.with_wt = with_wt;
    f.aux = aux_stream;
    return hip_status(lce::launch_flce(f, stream), "lce_flce_fwd_bwd launch");
}

size_t lce_flce_stats_bytes(int64_t n, int64_t V) {
    if (n < 0 || V < 1) return 0;
    return lce::flce_stats_bytes(n, V);
}

lce_status lce_flce_forward(const void *hidden, const void *weight, const int64_t *labels, int64_t n, int64_t H,
                            int64_t V, int64_t ignore_index, float label_smoothing, float softcap,
                            lce_reduction reduction, float *loss_tok, float *loss_out, float *lse, float *one_minus_py,
                            float *logprob, float *entropy, int64_t *argmax_out, int64_t *counts, void *workspace,
                            size_t workspace_bytes, hipStream_t stream) {
    const char *fn = "lce_flce_forward";
    lce_status st = check_flce_resident(fn, hidden, weight, labels, n, H, V, label_smoothing, softcap, reduction);
    if (st != LCE_OK) return st;
    if (!counts) return fail(LCE_ERR_INVALID_ARG, "%s: counts is required", fn);
    if (n > 0 && (!loss_tok || !lse || !one_minus_py))
        return fail(LCE_ERR_INVALID_ARG, "%s: loss_tok, lse and one_minus_py are required", fn);
    const size_t need = lce::flce_stats_bytes(n, V);
    if (n > 0 && (!workspace || workspace_bytes < need))
        return fail(LCE_ERR_INVALID_ARG, "%s: workspace_bytes %zu < minimum %zu", fn, workspace_bytes, need);
    if (n > 0 && !is_aligned(workspace, 256))
        return fail(LCE_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", fn);
    lce::FlceFwdArgs f;
    f.hidden = hidden;
    f.weight = weight;
    f.labels = labels;
    f.n = n;
    f.H = H;
    f.V = V;
    f.ignore_index = ignore_index;
    f.eps = label_smoothing;
    f.softcap = softcap;
    f.reduction = static_cast<int>(reduction);
    f.lse = lse;
    f.q = one_minus_py;
    f.loss_tok = loss_tok;
    f.loss_out = loss_out;
    f.logp = logprob;
    f.ent = entropy;
    f.argmax_out = argmax_out;
    f.counts = counts;
    f.workspace = workspace;
    return hip_status(lce::launch_flce_forward(f, stream), "lce_flce_forward launch");
}

lce_status lce_flce_backward(const void *hidden, const void *weight, const int64_t *labels, int64_t n, int64_t H,
                             int64_t V, int64_t ignore_index, float label_smoothing, float softcap,
                             lce_reduction reduction, const float *grad_out, int64_t chunk_tokens, const float *lse,
                             const float *one_minus_py, const int64_t *counts, void *grad_hidden, float *grad_weight,
                             void *workspace, size_t workspace_bytes, hipStream_t stream, hipStream_t aux_stream) {
    const char *fn = "lce_flce_backward";
    lce_status st = check_flce_resident(fn, hidden, weight, labels, n, H, V, label_smoothing, softcap, reduction);
    if (st != LCE_OK) return st;
    if (chunk_tokens < 1) return fail(LCE_ERR_INVALID_ARG, "%s: chunk_tokens must be >= 1", fn);
    if (!grad_weight || !counts || !workspace)
        return fail(LCE_ERR_INVALID_ARG, "%s: grad_weight, counts and workspace are required", fn);
    if (n > 0 && (!grad_hidden || !lse || !one_minus_py))
        return fail(LCE_ERR_INVALID_ARG, "%s: grad_hidden, lse and one_minus_py are required", fn);
    if ((grad_hidden && !is_aligned(grad_hidden, 16)) || !is_aligned(grad_weight, 16))
        return fail(LCE_ERR_UNSUPPORTED, "%s: grad_hidden and grad_weight must be 16-byte aligned", fn);
    int64_t group = 1;
    bool with_wt = false;
    const bool fits = lce::flce_plan(n, H, V, chunk_tokens, workspace_bytes, &group, &with_wt);
    const size_t need = lce::flce_layout(n, H, V, chunk_tokens, 1, false).bytes;
    if (!fits)
        return fail(LCE_ERR_INVALID_ARG, "%s: workspace_bytes %zu < minimum %zu", fn, workspace_bytes, need);
    if (!is_aligned(workspace, 256)) return fail(LCE_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", fn);
    const int64_t C = chunk_tokens < n ? chunk_tokens : n;
    if (C > 0x7fffffffLL / 16 || static_cast<unsigned long long>(C) * V * 2 >= (1ull << 32))
        return fail(LCE_ERR_UNSUPPORTED, "%s: a chunk of gradients exceeds 4 GiB", fn);
    if (!with_wt && n > 0 && static_cast<unsigned long long>(V) * H * 2 >= (1ull << 32))
        return fail(LCE_ERR_UNSUPPORTED,
                    "%s: without room for W^T in the workspace the grad_hidden GEMM reads the weight in place, "
                    "which needs V * H * 2 < 4 GiB (V=%lld H=%lld); pass lce_flce_workspace_bytes() bytes", fn,
                    (long long)V, (long long)H);
    lce::FlceArgs f;
    f.hidden = hidden;
    f.weight = weight;
    f.labels = labels;
    f.n = n;
    f.H = H;
    f.V = V;
    f.chunk = chunk_tokens;
    f.ignore_index = ignore_index;
    f.eps = label_smoothing;
    f.softcap = softcap;
    f.reduction = static_cast<int>(reduction);
    f.grad_out = grad_out;
    f.loss_tok = nullptr;
    f.loss_out = nullptr;
    f.grad_hidden = grad_hidden;
    f.grad_weight = grad_weight;
    f.counts = const_cast<int64_t *>(counts);   // read only on this path
    f.workspace = workspace;
    f.group_chunks = group;
    f.with_wt = with_wt;
    f.lse = lse;
    f.q = one_minus_py;
    f.aux = aux_stream;
    return hip_status(lce::launch_flce(f, stream), "lce_flce_backward launch");
}

}  // extern "C"

// ---- around the cross-entropy: the final norm, the rules on logits, the matrix product -----------

namespace {

size_t dtype_bytes(lce_dtype t) { return t == LCE_F32 ? 4 : t == LCE_BF16 ? 2 : 1; }

bool f32_or_bf16(lce_dtype t) { return t == LCE_F32 || t == LCE_BF16; }

// A matrix operand: present if required, row stride >= width, aligned to its element.
lce_status check_matrix(const char *fn, const char *name, const void *p, int64_t ld, int64_t width, lce_dtype t,
                        bool required) {
    if (!p) return required ? fail(LCE_ERR_INVALID_ARG, "%s: %s is required", fn, name) : LCE_OK;
    if (ld < width)
        return fail(LCE_ERR_INVALID_ARG, "%s: the row stride of %s (%lld) must be >= %lld", fn, name, (long long)ld,
                    (long long)width);
    if (!is_aligned(p, dtype_bytes(t)))
        return fail(LCE_ERR_INVALID_ARG, "%s: %s must be %zu-byte aligned", fn, name, dtype_bytes(t));
    return LCE_OK;
}

// An output in the place of an input that every row or tile reads: some would read it overwritten.
lce_status check_apart(const char *fn, const char *out_name, const void *out, const char *in_name, const void *in) {
    return out && out == in ? fail(LCE_ERR_INVALID_ARG, "%s: %s must not be %s", fn, out_name, in_name) : LCE_OK;
}

// A residual in the place of the output: each value is read where it is written, if the rows are the same.
lce_status check_residual(const char *fn, const void *residual, int64_t ldr, const void *out, int64_t ldo, int64_t n) {
    return residual && residual == out && n > 1 && ldr != ldo
               ? fail(LCE_ERR_INVALID_ARG, "%s: a residual in the place of out must have its row stride (%lld, got %lld)", fn,
                      (long long)ldo, (long long)ldr)
               : LCE_OK;
}

lce_status check_norm_sizes(const char *fn, int64_t n, int64_t H, lce_dtype dtype, const void *weight,
                            lce_dtype weight_dtype, float weight_offset) {
    if (n < 0) return fail(LCE_ERR_INVALID_ARG, "%s: n must be >= 0 (got %lld)", fn, (long long)n);
    if (H < 1) return fail(LCE_ERR_INVALID_ARG, "%s: H must be >= 1 (got %lld)", fn, (long long)H);
    if (!f32_or_bf16(dtype)) return fail(LCE_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    if (weight && !f32_or_bf16(weight_dtype))
        return fail(LCE_ERR_INVALID_ARG, "%s: unknown weight dtype %d", fn, (int)weight_dtype);
    if (!isfinite(weight_offset))
        return fail(LCE_ERR_INVALID_ARG, "%s: weight_offset must be finite (got %g)", fn, (double)weight_offset);
    if (weight && !is_aligned(weight, dtype_bytes(weight_dtype)))
        return fail(LCE_ERR_INVALID_ARG, "%s: weight must be %zu-byte aligned", fn, dtype_bytes(weight_dtype));
    if (H > lce::kNormMaxH)
        return fail(LCE_ERR_UNSUPPORTED, "%s: H must be <= %lld (got %lld)", fn, (long long)lce::kNormMaxH, (long long)H);
    if (n > 0x7fffffffLL) return fail(LCE_ERR_UNSUPPORTED, "%s: n > 2^31-1", fn);
    return LCE_OK;
}

}  // namespace

extern "C" {

lce_status lce_rms_norm(const void *x, int64_t ldx, lce_dtype dtype, const void *residual, int64_t ldr,
                        const void *weight, lce_dtype weight_dtype, float weight_offset, float eps, int64_t n,
                        int64_t H, void *sum, int64_t lds, void *y, int64_t ldy, lce_dtype y_dtype, float *scale,
                        float *rstd, hipStream_t stream) {
    const char *fn = "lce_rms_norm";
    lce_status st = check_norm_sizes(fn, n, H, dtype, weight, weight_dtype, weight_offset);
    if (st != LCE_OK) return st;
    if (!(eps >= 0.0f) || isinf(eps))
        return fail(LCE_ERR_INVALID_ARG, "%s: eps must be finite and >= 0 (got %g)", fn, (double)eps);
    if (y_dtype != dtype && y_dtype != LCE_E4M3)
        return fail(LCE_ERR_INVALID_ARG, "%s: y must have the dtype of x or be e4m3 (got %d)", fn, (int)y_dtype);
    if (n == 0) return ok();
    if ((st = check_matrix(fn, "x", x, ldx, H, dtype, true)) != LCE_OK ||
        (st = check_matrix(fn, "residual", residual, ldr, H, dtype, false)) != LCE_OK ||
        (st = check_matrix(fn, "sum", sum, lds, H, dtype, false)) != LCE_OK ||
        (st = check_matrix(fn, "y", y, ldy, H, y_dtype, true)) != LCE_OK)
        return st;
    if (y_dtype == LCE_E4M3 && !scale)
        return fail(LCE_ERR_INVALID_ARG, "%s: scale is required for an e4m3 output", fn);
    if ((st = check_apart(fn, "y", y, "weight", weight)) != LCE_OK ||
        (st = check_apart(fn, "sum", sum, "weight", weight)) != LCE_OK ||
        (st = check_apart(fn, "rstd", rstd, "weight", weight)) != LCE_OK ||
        (st = check_apart(fn, "scale", y_dtype == LCE_E4M3 ? scale : nullptr, "weight", weight)) != LCE_OK)
        return st;
    lce::NormArgs a;
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.sum = sum;
    a.y = y;
    a.rstd = rstd;
    a.scale = scale;
    a.ldx = ldx;
    a.ldr = ldr;
    a.lds = lds;
    a.ldy = ldy;
    a.n = n;
    a.H = H;
    a.eps = eps;
    a.offset = weight_offset;
    a.weight_bf16 = weight_dtype == LCE_BF16;
    a.out8 = y_dtype == LCE_E4M3;
    return hip_status(lce::launch_rms_norm(a, dtype == LCE_BF16, stream), "lce_rms_norm launch");
}

size_t lce_rms_norm_workspace_bytes(int64_t n, int64_t H) {
    if (n < 0 || H < 1 || H > lce::kNormMaxH) return 0;
    return static_cast<size_t>(n < lce::kNormMaxGroups ? n : lce::kNormMaxGroups) * static_cast<size_t>(H) * 4;
}

lce_status lce_rms_norm_backward(const void *grad_y, int64_t ldg, const void *s, int64_t lds, lce_dtype dtype,
                                 const void *weight, lce_dtype weight_dtype, float weight_offset, const float *rstd,
                                 const void *grad_sum, int64_t ldgs, int64_t n, int64_t H, void *grad_x, int64_t ldgx,
                                 void *grad_weight, lce_dtype grad_weight_dtype, void *workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
    const char *fn = "lce_rms_norm_backward";
    lce_status st = check_norm_sizes(fn, n, H, dtype, weight, weight_dtype, weight_offset);
    if (st != LCE_OK) return st;
    if (grad_weight && !f32_or_bf16(grad_weight_dtype))
        return fail(LCE_ERR_INVALID_ARG, "%s: unknown grad_weight dtype %d", fn, (int)grad_weight_dtype);
    if (grad_weight && !is_aligned(grad_weight, dtype_bytes(grad_weight_dtype)))
        return fail(LCE_ERR_INVALID_ARG, "%s: grad_weight must be %zu-byte aligned", fn, dtype_bytes(grad_weight_dtype));
    if (n > 0) {
        if ((st = check_matrix(fn, "grad_y", grad_y, ldg, H, dtype, true)) != LCE_OK ||
            (st = check_matrix(fn, "s", s, lds, H, dtype, true)) != LCE_OK ||
            (st = check_matrix(fn, "grad_sum", grad_sum, ldgs, H, dtype, false)) != LCE_OK ||
            (st = check_matrix(fn, "grad_x", grad_x, ldgx, H, dtype, true)) != LCE_OK)
            return st;
        if (!rstd) return fail(LCE_ERR_INVALID_ARG, "%s: rstd is required", fn);
        if (grad_weight) {
            const size_t need = lce_rms_norm_workspace_bytes(n, H);
            if (!workspace || workspace_bytes < need)
                return fail(LCE_ERR_INVALID_ARG, "%s: workspace_bytes %zu < minimum %zu", fn, workspace_bytes, need);
            if (!is_aligned(workspace, 16))
                return fail(LCE_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", fn);
        }
        if ((st = check_apart(fn, "grad_x", grad_x, "weight", weight)) != LCE_OK) return st;
    }
    lce::NormGradArgs a;
    a.gy = grad_y;
    a.s = s;
    a.weight = weight;
    a.gs = grad_sum;
    a.rstd = rstd;
    a.gx = grad_x;
    a.gw = grad_weight;
    a.part = static_cast<float *>(workspace);
    a.ldg = ldg;
    a.lds = lds;
    a.ldgs = ldgs;
    a.ldgx = ldgx;
    a.n = n;
    a.H = H;
    a.offset = weight_offset;
    a.weight_bf16 = weight_dtype == LCE_BF16;
    a.gw_bf16 = grad_weight_dtype == LCE_BF16;
    return hip_status(lce::launch_rms_norm_backward(a, dtype == LCE_BF16, stream), "lce_rms_norm_backward launch");
}

lce_status lce_logits_process(const void *logits, int64_t ldx, lce_dtype dtype, int64_t n, int64_t V,
                              const void *history, int64_t ldh, int64_t L, const int64_t *history_lens,
                              const int64_t *prompt_lens, const void *bias_ids, int64_t ldbi, const float *bias_values,
                              int64_t ldbv, int64_t B, int ids_are_64, const float *repetition, const float *presence,
                              const float *frequency, const float *temperature, const uint32_t *allowed, int64_t ldm,
                              int64_t mask_count, const int64_t *mask_rows, float mask_value, float softcap, void *out,
                              int64_t ldo, hipStream_t stream) {
    const char *fn = "lce_logits_process";
    lce_status st;
    if (n < 0) return fail(LCE_ERR_INVALID_ARG, "%s: n must be >= 0 (got %lld)", fn, (long long)n);
    if (V < 1) return fail(LCE_ERR_INVALID_ARG, "%s: V must be >= 1 (got %lld)", fn, (long long)V);
    if (!f32_or_bf16(dtype)) return fail(LCE_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    if (!(softcap >= 0.0f) || isinf(softcap))
        return fail(LCE_ERR_INVALID_ARG, "%s: softcap must be finite and >= 0 (got %g)", fn, (double)softcap);
    if (isnan(mask_value)) return fail(LCE_ERR_INVALID_ARG, "%s: mask_value must not be NaN", fn);
    const size_t idb = ids_are_64 ? 8 : 4;
    if (history) {
        if (L < 0) return fail(LCE_ERR_INVALID_ARG, "%s: L must be >= 0 (got %lld)", fn, (long long)L);
        if (ldh != 0 && ldh < L)
            return fail(LCE_ERR_INVALID_ARG, "%s: the row stride of history (%lld) must be 0 or >= %lld", fn,
                        (long long)ldh, (long long)L);
        if (!is_aligned(history, idb)) return fail(LCE_ERR_INVALID_ARG, "%s: history must be %zu-byte aligned", fn, idb);
    }
    if (!bias_ids != !bias_values)
        return fail(LCE_ERR_INVALID_ARG, "%s: bias_ids and bias_values go together", fn);
    if (bias_ids) {
        if (B < 0) return fail(LCE_ERR_INVALID_ARG, "%s: B must be >= 0 (got %lld)", fn, (long long)B);
        if ((ldbi != 0 && ldbi < B) || (ldbv != 0 && ldbv < B))
            return fail(LCE_ERR_INVALID_ARG, "%s: the row strides of the biases must be 0 or >= %lld", fn, (long long)B);
        if (!is_aligned(bias_ids, idb) || !is_aligned(bias_values, 4))
            return fail(LCE_ERR_INVALID_ARG, "%s: bias_ids and bias_values must be aligned to their elements", fn);
    }
    if (allowed) {
        const int64_t words = (V + 31) / 32;
        if (mask_count < 0) return fail(LCE_ERR_INVALID_ARG, "%s: mask_count must be >= 0", fn);
        if (ldm < words)
            return fail(LCE_ERR_INVALID_ARG, "%s: the row stride of allowed (%lld) must be >= %lld words", fn,
                        (long long)ldm, (long long)words);
        if (!mask_rows && mask_count < n)
            return fail(LCE_ERR_INVALID_ARG, "%s: without mask_rows every row needs a mask (%lld of %lld)", fn,
                        (long long)mask_count, (long long)n);
        if (!is_aligned(allowed, 4)) return fail(LCE_ERR_INVALID_ARG, "%s: allowed must be 4-byte aligned", fn);
    }
    // column arithmetic is 32-bit, and a count fits the low 31 bits of its word
    if (V > 0x7fffffffLL - 65536) return fail(LCE_ERR_UNSUPPORTED, "%s: V must be < 2^31 - 65536", fn);
    if ((history && L > 0x7fffffffLL) || (bias_ids && B > 0x7fffffffLL))
        return fail(LCE_ERR_UNSUPPORTED, "%s: L and B must be < 2^31", fn);
    if (n > 0x7fffffffLL) return fail(LCE_ERR_UNSUPPORTED, "%s: n > 2^31-1", fn);
    if (n == 0) return ok();
    if ((st = check_matrix(fn, "logits", logits, ldx, V, dtype, true)) != LCE_OK ||
        (st = check_matrix(fn, "out", out, ldo, V, dtype, true)) != LCE_OK ||
        (st = check_apart(fn, "out", out, "bias_values", bias_values)) != LCE_OK ||
        (st = check_apart(fn, "out", out, "repetition", repetition)) != LCE_OK ||
        (st = check_apart(fn, "out", out, "presence", presence)) != LCE_OK ||
        (st = check_apart(fn, "out", out, "frequency", frequency)) != LCE_OK ||
        (st = check_apart(fn, "out", out, "temperature", temperature)) != LCE_OK)
        return st;
    lce::RulesArgs a;
    a.logits = logits;
    a.out = out;
    a.ldx = ldx;
    a.ldo = ldo;
    a.n = n;
    a.V = V;
    a.history = L > 0 ? history : nullptr;
    a.ldh = ldh;
    a.L = L;
    a.history_lens = history_lens;
    a.prompt_lens = prompt_lens;
    a.bias_ids = B > 0 ? bias_ids : nullptr;
    a.bias_values = bias_values;
    a.ldbi = ldbi;
    a.ldbv = ldbv;
    a.B = B;
    a.id64 = ids_are_64 != 0;
    a.repetition = repetition;
    a.presence = presence;
    a.frequency = frequency;
    a.temperature = temperature;
    a.allowed = allowed;
    a.ldm = ldm;
    a.R = mask_count;
    a.mask_rows = mask_rows;
    a.mask_value = mask_value;
    a.softcap = softcap;
    return hip_status(lce::launch_logits_process(a, dtype == LCE_BF16, stream), "lce_logits_process launch");
}

}  // extern "C"

namespace {

// Sizes and operands both directions of the product share.  es: bytes of an operand's element.
lce_status check_linear(const char *fn, const void *x, int64_t ldx, const void *weight, int64_t ldw, int64_t n, int64_t K,
                        int64_t M, int act, int64_t es) {
    if (n < 0) return fail(LCE_ERR_INVALID_ARG, "%s: n must be >= 0 (got %lld)", fn, (long long)n);
    if (K < 1) return fail(LCE_ERR_INVALID_ARG, "%s: K must be >= 1 (got %lld)", fn, (long long)K);
    if (M < 1) return fail(LCE_ERR_INVALID_ARG, "%s: M must be >= 1 (got %lld)", fn, (long long)M);
    if (act < LCE_ACT_NONE || act > LCE_ACT_SILU) return fail(LCE_ERR_INVALID_ARG, "%s: unknown activation %d", fn, act);
    if (!weight) return fail(LCE_ERR_INVALID_ARG, "%s: weight is required", fn);
    if (n > 0 && !x) return fail(LCE_ERR_INVALID_ARG, "%s: x is required", fn);
    if (ldx < K || ldw < K)
        return fail(LCE_ERR_INVALID_ARG, "%s: the row strides of x (%lld) and weight (%lld) must be >= %lld", fn,
                    (long long)ldx, (long long)ldw, (long long)K);
    const int64_t unit = 16 / es;
    if (K % unit || ldx % unit || ldw % unit)
        return fail(LCE_ERR_UNSUPPORTED, "%s: K and the row strides of x and weight must be multiples of %lld (16 bytes)",
                    fn, (long long)unit);
    if ((x && !is_aligned(x, 16)) || !is_aligned(weight, 16))
        return fail(LCE_ERR_UNSUPPORTED, "%s: x and weight must be 16-byte aligned", fn);
    if (ldx > lce::kLinearMaxStride / es || ldw > lce::kLinearMaxStride / es || n > 0x7fffffffLL / 256 || M > 0x7fffffffLL / 256)
        return fail(LCE_ERR_UNSUPPORTED, "%s: 256 rows of x or weight exceed 4 GiB, or n or M >= 2^23", fn);
    return LCE_OK;
}

}  // namespace

extern "C" {

size_t lce_linear_workspace_bytes(int64_t n, int64_t K, int64_t M, lce_dtype in_dtype) {
    if (n < 0 || K < 1 || M < 1) return 0;
    return lce::linear_workspace_bytes(n, K, M, in_dtype == LCE_E4M3);
}

lce_status lce_linear(const void *x, int64_t ldx, const void *weight, int64_t ldw, lce_dtype in_dtype,
                      const float *scale_x, const float *scale_w, const void *bias, lce_dtype bias_dtype,
                      lce_activation act, const void *residual, int64_t ldr, int64_t n, int64_t K, int64_t M, void *out,
                      int64_t ldo, lce_dtype out_dtype, void *preact, int64_t ldp, void *workspace,
                      size_t workspace_bytes, hipStream_t stream) {
    const char *fn = "lce_linear";
    if (in_dtype != LCE_BF16 && in_dtype != LCE_E4M3)
        return fail(LCE_ERR_INVALID_ARG, "%s: x and weight must be bf16 or e4m3 (got dtype %d)", fn, (int)in_dtype);
    lce_status st = check_linear(fn, x, ldx, weight, ldw, n, K, M, act, in_dtype == LCE_E4M3 ? 1 : 2);
    if (st != LCE_OK) return st;
    if (in_dtype == LCE_BF16 && (scale_x || scale_w))
        return fail(LCE_ERR_INVALID_ARG, "%s: scales go with e4m3 operands", fn);
    if (!f32_or_bf16(out_dtype)) return fail(LCE_ERR_INVALID_ARG, "%s: unknown output dtype %d", fn, (int)out_dtype);
    if (in_dtype == LCE_E4M3 && out_dtype != LCE_BF16)
        return fail(LCE_ERR_UNSUPPORTED, "%s: e4m3 operands give a bf16 output", fn);
    if (bias && !f32_or_bf16(bias_dtype)) return fail(LCE_ERR_INVALID_ARG, "%s: unknown bias dtype %d", fn, (int)bias_dtype);
    if (bias && !is_aligned(bias, dtype_bytes(bias_dtype)))
        return fail(LCE_ERR_INVALID_ARG, "%s: bias must be %zu-byte aligned", fn, dtype_bytes(bias_dtype));
    if (n == 0) return ok();
    if ((st = check_matrix(fn, "residual", residual, ldr, M, out_dtype, false)) != LCE_OK ||
        (st = check_matrix(fn, "out", out, ldo, M, out_dtype, true)) != LCE_OK ||
        (st = check_matrix(fn, "preact", preact, ldp, M, LCE_BF16, false)) != LCE_OK)
        return st;
    const size_t need = lce::linear_workspace_bytes(n, K, M, in_dtype == LCE_E4M3);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(LCE_ERR_INVALID_ARG, "%s: workspace_bytes %zu < minimum %zu", fn, workspace_bytes, need);
    if (need > 0 && !is_aligned(workspace, 16))
        return fail(LCE_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", fn);
    // every tile reads whole rows of x and weight; the residual is read after the pre-activation is written
    if (out == x || out == weight || (preact && (preact == x || preact == weight)))
        return fail(LCE_ERR_INVALID_ARG, "%s: out and preact must not be x or weight", fn);
    if (preact && (preact == residual || preact == out))
        return fail(LCE_ERR_INVALID_ARG, "%s: preact must not be residual or out", fn);
    if ((st = check_apart(fn, "out", out, "bias", bias)) != LCE_OK ||
        (st = check_apart(fn, "preact", preact, "bias", bias)) != LCE_OK ||
        (st = check_residual(fn, residual, ldr, out, ldo, n)) != LCE_OK)
        return st;
    lce::LinearArgs a{};
    a.x = x;
    a.weight = weight;
    a.ldx = ldx;
    a.ldw = ldw;
    a.n = n;
    a.K = K;
    a.M = M;
    a.fp8 = in_dtype == LCE_E4M3;
    a.scale_x = scale_x;
    a.scale_w = scale_w;
    a.bias = bias;
    a.bias_bf16 = bias_dtype == LCE_BF16;
    a.act = act;
    a.residual = residual;
    a.ldr = ldr;
    a.out = out;
    a.ldo = ldo;
    a.out_bf16 = out_dtype == LCE_BF16;
    a.preact = preact;
    a.ldp = ldp;
    a.part = static_cast<float *>(workspace);
    return hip_status(lce::launch_linear(a, stream), "lce_linear launch");
}

size_t lce_linear_backward_workspace_bytes(int64_t n, int64_t K, int64_t M) {
    if (n < 0 || K < 1 || M < 1) return 0;
    return lce::linear_backward_workspace_bytes(n, K, M);
}

lce_status lce_linear_backward(const void *grad_out, int64_t ldg, lce_dtype grad_dtype, const void *x, int64_t ldx,
                               const void *weight, int64_t ldw, const void *preact, int64_t ldp, lce_activation act,
                               int64_t n, int64_t K, int64_t M, void *grad_x, int64_t ldgx, void *grad_weight,
                               lce_dtype grad_weight_dtype, void *grad_bias, lce_dtype grad_bias_dtype, void *workspace,
                               size_t workspace_bytes, hipStream_t stream) {
    const char *fn = "lce_linear_backward";
    lce_status st = check_linear(fn, x, ldx, weight, ldw, n, K, M, act, 2);
    if (st != LCE_OK) return st;
    if (M % 8) return fail(LCE_ERR_UNSUPPORTED, "%s: M must be a multiple of 8 (got %lld)", fn, (long long)M);
    if (K > 0x7fffffffLL / 256) return fail(LCE_ERR_UNSUPPORTED, "%s: K >= 2^23", fn);
    // n and M are row lengths of what the products read: the limit check_linear puts on ldx and ldw
    if (n > (1 << 23) - 512 || M > (1 << 23) - 512)
        return fail(LCE_ERR_UNSUPPORTED, "%s: n and M must be <= 2^23 - 512 (got %lld, %lld)", fn, (long long)n, (long long)M);
    // the transposes' workgroups, of 128 x 64 values each, are one launch of fewer than 2^32 threads
    if ((n / 128 + 1) * ((M + K) / 64 + 2) + (M / 128 + 1) * (K / 64 + 1) >= (int64_t(1) << 23))
        return fail(LCE_ERR_UNSUPPORTED, "%s: n (M + K) + M K must be below 2^36", fn);
    if (!f32_or_bf16(grad_dtype)) return fail(LCE_ERR_INVALID_ARG, "%s: unknown grad_out dtype %d", fn, (int)grad_dtype);
    if (grad_weight && !f32_or_bf16(grad_weight_dtype))
        return fail(LCE_ERR_INVALID_ARG, "%s: unknown grad_weight dtype %d", fn, (int)grad_weight_dtype);
    if (grad_bias && !f32_or_bf16(grad_bias_dtype))
        return fail(LCE_ERR_INVALID_ARG, "%s: unknown grad_bias dtype %d", fn, (int)grad_bias_dtype);
    if (n > 0) {
        if ((st = check_matrix(fn, "grad_out", grad_out, ldg, M, grad_dtype, true)) != LCE_OK ||
            (st = check_matrix(fn, "preact", preact, ldp, M, LCE_BF16, act != LCE_ACT_NONE)) != LCE_OK ||
            (st = check_matrix(fn, "grad_x", grad_x, ldgx, K, LCE_BF16, false)) != LCE_OK)
            return st;
    }
    if (grad_x && (!is_aligned(grad_x, 16) || ldgx % 8))
        return fail(LCE_ERR_UNSUPPORTED, "%s: grad_x must be 16-byte aligned with a row stride of whole 16 bytes", fn);
    if (grad_weight && !is_aligned(grad_weight, 16))
        return fail(LCE_ERR_UNSUPPORTED, "%s: grad_weight must be 16-byte aligned", fn);
    if (grad_bias && !is_aligned(grad_bias, dtype_bytes(grad_bias_dtype)))
        return fail(LCE_ERR_INVALID_ARG, "%s: grad_bias must be %zu-byte aligned", fn, dtype_bytes(grad_bias_dtype));
    const size_t need = lce::linear_backward_workspace_bytes(n, K, M);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(LCE_ERR_INVALID_ARG, "%s: workspace_bytes %zu < minimum %zu", fn, workspace_bytes, need);
    if (need > 0 && !is_aligned(workspace, 256))
        return fail(LCE_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", fn);
    if ((st = check_apart(fn, "grad_bias", grad_bias, "grad_out", grad_out)) != LCE_OK ||
        (st = check_apart(fn, "grad_bias", grad_bias, "preact", preact)) != LCE_OK ||
        (st = check_apart(fn, "grad_bias", grad_bias, "x", x)) != LCE_OK ||
        (st = check_apart(fn, "grad_bias", grad_bias, "weight", weight)) != LCE_OK)
        return st;
    lce::LinearGradArgs a{};
    a.grad_out = grad_out;
    a.ldg = ldg;
    a.grad_bf16 = grad_dtype == LCE_BF16;
    a.x = x;
    a.weight = weight;
    a.ldx = ldx;
    a.ldw = ldw;
    a.preact = preact;
    a.ldp = ldp;
    a.act = act;
    a.n = n;
    a.K = K;
    a.M = M;
    a.grad_x = grad_x;
    a.ldgx = ldgx;
    a.grad_weight = grad_weight;
    a.grad_weight_bf16 = grad_weight_dtype == LCE_BF16;
    a.grad_bias = grad_bias;
    a.grad_bias_bf16 = grad_bias_dtype == LCE_BF16;
    a.workspace = workspace;
    return hip_status(lce::launch_linear_backward(a, stream), "lce_linear_backward launch");
}

}  // extern "C"

namespace {

// Strides of a [rows, cols] array of scales, no two at one place where it is written.
lce_status check_scale(const char *fn, const char *name, const void *p, int64_t s_row, int64_t s_col, int64_t rows,
                       int64_t cols, lce_dtype dtype, bool written) {
    if (dtype != LCE_F32 && dtype != LCE_E8M0)
        return fail(LCE_ERR_INVALID_ARG, "%s: %s must be fp32 or e8m0 (got dtype %d)", fn, name, (int)dtype);
    if (!p) return fail(LCE_ERR_INVALID_ARG, "%s: %s is required", fn, name);
    if (s_row < 0 || s_col < 0) return fail(LCE_ERR_INVALID_ARG, "%s: the strides of %s must be >= 0", fn, name);
    if (s_row > INT64_MAX / 8 / rows || s_col > INT64_MAX / 8 / cols)
        return fail(LCE_ERR_INVALID_ARG, "%s: the strides of %s are too large", fn, name);
    const bool by_row = (cols <= 1 || s_col >= 1) && (rows <= 1 || s_row >= (cols - 1) * s_col + 1);
    const bool by_col = (rows <= 1 || s_row >= 1) && (cols <= 1 || s_col >= (rows - 1) * s_row + 1);
    if (written && !by_row && !by_col)
        return fail(LCE_ERR_INVALID_ARG, "%s: the strides of %s (%lld, %lld) put two scales at one place", fn, name,
                    (long long)s_row, (long long)s_col);
    if (dtype == LCE_F32 && !is_aligned(p, 4)) return fail(LCE_ERR_INVALID_ARG, "%s: %s must be 4-byte aligned", fn, name);
    return LCE_OK;
}

// An e4m3 matrix as the product reads it.
lce_status check_blocked(const char *fn, const char *name, const void *p, int64_t ld, int64_t K) {
    if (!p) return fail(LCE_ERR_INVALID_ARG, "%s: %s is required", fn, name);
    if (ld < K)
        return fail(LCE_ERR_INVALID_ARG, "%s: the row stride of %s (%lld) must be >= %lld", fn, name, (long long)ld, (long long)K);
    if (ld % 16 || !is_aligned(p, 16))
        return fail(LCE_ERR_UNSUPPORTED, "%s: %s must be 16-byte aligned with a row stride of whole 16 bytes", fn, name);
    if (ld > lce::kLinearMaxStride)
        return fail(LCE_ERR_UNSUPPORTED, "%s: 256 rows of %s exceed 4 GiB", fn, name);
    return LCE_OK;
}

lce_status check_blocks_sizes(const char *fn, int64_t n, int64_t K, int64_t M) {
    if (n < 0) return fail(LCE_ERR_INVALID_ARG, "%s: n must be >= 0 (got %lld)", fn, (long long)n);
    if (K < 1) return fail(LCE_ERR_INVALID_ARG, "%s: K must be >= 1 (got %lld)", fn, (long long)K);
    if (M < 1) return fail(LCE_ERR_INVALID_ARG, "%s: M must be >= 1 (got %lld)", fn, (long long)M);
    if (n > 0x7fffffffLL / 256 || M > 0x7fffffffLL / 256) return fail(LCE_ERR_UNSUPPORTED, "%s: n or M >= 2^23", fn);
    return LCE_OK;
}

lce_status check_training_sizes(const char *fn, int64_t n, int64_t K, int64_t M) {
    const lce_status st = check_blocks_sizes(fn, n, K, M);
    if (st != LCE_OK) return st;
    if (K > 0x7fffffffLL / 256) return fail(LCE_ERR_UNSUPPORTED, "%s: K >= 2^23", fn);
    if (n > (1 << 23) - 1024 || M > (1 << 23) - 1024)   // row lengths of what the products read
        return fail(LCE_ERR_UNSUPPORTED, "%s: n and M must be <= 2^23 - 1024 (got %lld, %lld)", fn, (long long)n, (long long)M);
    return LCE_OK;
}

// whether 128 x 128 blocks of [n, K] number fewer than 2^24
bool few_blocks(int64_t n, int64_t K) {
    const int64_t rows = n / 128 + 1, cols = K / 128 + 1;
    return rows < (int64_t(1) << 24) && cols < (int64_t(1) << 24) && rows * cols < (int64_t(1) << 24);
}

}  // namespace

extern "C" {

lce_status lce_quantize_blocks(const void *x, int64_t ldx, lce_dtype dtype, int64_t n, int64_t K, void *values,
                               int64_t ldv, lce_blocks blocks, void *scale, int64_t s_row, int64_t s_col,
                               void *values_t, int64_t ldvt, lce_blocks blocks_t, void *scale_t, int64_t st_row,
                               int64_t st_col, lce_dtype scale_dtype, hipStream_t stream) {
    const char *fn = "lce_quantize_blocks";
    if (n < 0) return fail(LCE_ERR_INVALID_ARG, "%s: n must be >= 0 (got %lld)", fn, (long long)n);
    if (K < 1) return fail(LCE_ERR_INVALID_ARG, "%s: K must be >= 1 (got %lld)", fn, (long long)K);
    if (!f32_or_bf16(dtype)) return fail(LCE_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    for (int b : {(int)blocks, (int)blocks_t})
        if (b != LCE_BLOCKS_ROW && b != LCE_BLOCKS_TILE) return fail(LCE_ERR_INVALID_ARG, "%s: unknown blocks %d", fn, b);
    if (!few_blocks(n, K)) return fail(LCE_ERR_UNSUPPORTED, "%s: 2^24 or more blocks of 128 x 128", fn);
    if (n == 0) return ok();
    if (!values && !values_t) return fail(LCE_ERR_INVALID_ARG, "%s: values or values_t is required", fn);
    const int64_t bn = (n + 127) / 128, bk = (K + 127) / 128;
    lce_status st;
    if ((st = check_matrix(fn, "x", x, ldx, K, dtype, true)) != LCE_OK ||
        (st = check_matrix(fn, "values", values, ldv, K, LCE_E4M3, false)) != LCE_OK ||
        (st = check_matrix(fn, "values_t", values_t, ldvt, n, LCE_E4M3, false)) != LCE_OK)
        return st;
    if (values && (st = check_scale(fn, "scale", scale, s_row, s_col, blocks == LCE_BLOCKS_TILE ? bn : n, bk, scale_dtype, true)) != LCE_OK)
        return st;
    if (values_t && (st = check_scale(fn, "scale_t", scale_t, st_row, st_col, blocks_t == LCE_BLOCKS_TILE ? bk : K, bn, scale_dtype, true)) != LCE_OK)
        return st;
    const void *outs[4] = {values, values ? scale : nullptr, values_t, values_t ? scale_t : nullptr};
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (outs[i] && outs[i] == outs[j]) return fail(LCE_ERR_INVALID_ARG, "%s: two outputs are the same buffer", fn);
    for (const void *o : outs)
        if (o == x) return fail(LCE_ERR_INVALID_ARG, "%s: an output must not be x", fn);
    lce::QuantizeArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.n = n;
    a.K = K;
    const bool e8m0 = scale_dtype == LCE_E8M0;
    a.q = {static_cast<unsigned char *>(values), ldv, scale, s_row, s_col, blocks == LCE_BLOCKS_TILE, e8m0};
    a.qt = {static_cast<unsigned char *>(values_t), ldvt, scale_t, st_row, st_col, blocks_t == LCE_BLOCKS_TILE, e8m0};
    return hip_status(lce::launch_quantize_blocks(a, dtype == LCE_BF16, stream), "lce_quantize_blocks launch");
}

size_t lce_linear_blocks_workspace_bytes(int64_t n, int64_t K, int64_t M) {
    if (check_blocks_sizes("lce_linear_blocks_workspace_bytes", n, K, M) != LCE_OK || K > lce::kLinearMaxStride) return 0;
    return lce::linear_blocks_workspace_bytes(n, K, M);
}

lce_status lce_linear_blocks(const void *x, int64_t ldx, const void *scale_x, int64_t sx_row, int64_t sx_col,
                             lce_dtype scale_x_dtype, const void *weight, int64_t ldw, const void *scale_w,
                             int64_t sw_row, int64_t sw_col, lce_dtype scale_w_dtype, const void *bias,
                             lce_dtype bias_dtype, lce_activation act, const void *residual, int64_t ldr, int64_t n,
                             int64_t K, int64_t M, void *out, int64_t ldo, void *preact, int64_t ldp, void *workspace,
                             size_t workspace_bytes, hipStream_t stream) {
    const char *fn = "lce_linear_blocks";
    lce_status st = check_blocks_sizes(fn, n, K, M);
    if (st != LCE_OK) return st;
    if (act < LCE_ACT_NONE || act > LCE_ACT_SILU) return fail(LCE_ERR_INVALID_ARG, "%s: unknown activation %d", fn, act);
    if (bias && !f32_or_bf16(bias_dtype)) return fail(LCE_ERR_INVALID_ARG, "%s: unknown bias dtype %d", fn, (int)bias_dtype);
    if (bias && !is_aligned(bias, dtype_bytes(bias_dtype)))
        return fail(LCE_ERR_INVALID_ARG, "%s: bias must be %zu-byte aligned", fn, dtype_bytes(bias_dtype));
    if (n == 0) return ok();
    const int64_t bk = (K + 127) / 128;
    if ((st = check_blocked(fn, "x", x, ldx, K)) != LCE_OK || (st = check_blocked(fn, "weight", weight, ldw, K)) != LCE_OK ||
        (st = check_scale(fn, "scale_x", scale_x, sx_row, sx_col, n, bk, scale_x_dtype, false)) != LCE_OK ||
        (st = check_scale(fn, "scale_w", scale_w, sw_row, sw_col, (M + 127) / 128, bk, scale_w_dtype, false)) != LCE_OK ||
        (st = check_matrix(fn, "residual", residual, ldr, M, LCE_BF16, false)) != LCE_OK ||
        (st = check_matrix(fn, "out", out, ldo, M, LCE_BF16, true)) != LCE_OK ||
        (st = check_matrix(fn, "preact", preact, ldp, M, LCE_BF16, false)) != LCE_OK)
        return st;
    const size_t need = lce::linear_blocks_workspace_bytes(n, K, M);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(LCE_ERR_INVALID_ARG, "%s: workspace_bytes %zu < minimum %zu", fn, workspace_bytes, need);
    if (need > 0 && !is_aligned(workspace, 16))
        return fail(LCE_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", fn);
    for (const void *o : {static_cast<const void *>(out), static_cast<const void *>(preact)})
        if (o && (o == x || o == weight || o == scale_x || o == scale_w))
            return fail(LCE_ERR_INVALID_ARG, "%s: out and preact must not be x, weight or a scale", fn);
    if (preact && (preact == residual || preact == out))
        return fail(LCE_ERR_INVALID_ARG, "%s: preact must not be residual or out", fn);
    if ((st = check_apart(fn, "out", out, "bias", bias)) != LCE_OK ||
        (st = check_apart(fn, "preact", preact, "bias", bias)) != LCE_OK ||
        (st = check_residual(fn, residual, ldr, out, ldo, n)) != LCE_OK)
        return st;
    lce::BlocksArgs a{};
    a.x = x;
    a.weight = weight;
    a.ldx = ldx;
    a.ldw = ldw;
    a.n = n;
    a.K = K;
    a.M = M;
    a.sx = {scale_x, sx_row, sx_col, scale_x_dtype == LCE_E8M0};
    a.sw = {scale_w, sw_row, sw_col, scale_w_dtype == LCE_E8M0};
    a.bias = bias;
    a.bias_bf16 = bias_dtype == LCE_BF16;
    a.act = act;
    a.residual = residual;
    a.ldr = ldr;
    a.out = out;
    a.ldo = ldo;
    a.preact = preact;
    a.ldp = ldp;
    a.part = static_cast<float *>(workspace);
    return hip_status(lce::launch_linear_blocks(a, stream), "lce_linear_blocks launch");
}

size_t lce_linear_blocks_forward_workspace_bytes(int64_t n, int64_t K, int64_t M) {
    if (check_training_sizes("lce_linear_blocks_forward_workspace_bytes", n, K, M) != LCE_OK) return 0;
    return lce::linear_blocks_forward_workspace_bytes(n, K, M);
}

lce_status lce_linear_blocks_forward(const void *x, int64_t ldx, const void *weight, int64_t ldw, const void *bias,
                                     lce_dtype bias_dtype, const void *residual, int64_t ldr, int64_t n, int64_t K,
                                     int64_t M, void *out, int64_t ldo, void *xt, int64_t ldxt, void *scale_xt,
                                     void *wt, int64_t ldwt, void *scale_wt, void *workspace, size_t workspace_bytes,
                                     hipStream_t stream) {
    const char *fn = "lce_linear_blocks_forward";
    lce_status st = check_training_sizes(fn, n, K, M);
    if (st != LCE_OK) return st;
    // both matrices are quantised in one launch
    if (!few_blocks(n, K) || !few_blocks(M, K) || ((n + 127) / 128 + (M + 127) / 128) * ((K + 127) / 128) >= (int64_t(1) << 24))
        return fail(LCE_ERR_UNSUPPORTED, "%s: 2^24 or more blocks of 128 x 128 in x and weight", fn);
    if (bias && !f32_or_bf16(bias_dtype)) return fail(LCE_ERR_INVALID_ARG, "%s: unknown bias dtype %d", fn, (int)bias_dtype);
    if (bias && !is_aligned(bias, dtype_bytes(bias_dtype)))
        return fail(LCE_ERR_INVALID_ARG, "%s: bias must be %zu-byte aligned", fn, dtype_bytes(bias_dtype));
    if (K > lce::kLinearMaxStride - 16) return fail(LCE_ERR_UNSUPPORTED, "%s: 256 rows of K values exceed 4 GiB", fn);
    if ((st = check_matrix(fn, "x", x, ldx, K, LCE_BF16, n > 0)) != LCE_OK ||
        (st = check_matrix(fn, "weight", weight, ldw, K, LCE_BF16, true)) != LCE_OK ||
        (st = check_matrix(fn, "residual", residual, ldr, M, LCE_BF16, false)) != LCE_OK ||
        (st = check_matrix(fn, "out", out, ldo, M, LCE_BF16, n > 0)) != LCE_OK)
        return st;
    if (n == 0) xt = out = nullptr;   // nothing of them is written
    if ((xt && ((st = check_blocked(fn, "xt", xt, ldxt, n)) != LCE_OK ||
                (st = check_scale(fn, "scale_xt", scale_xt, 1, 1, 1, 1, LCE_E8M0, true)) != LCE_OK)) ||
        (wt && ((st = check_blocked(fn, "wt", wt, ldwt, M)) != LCE_OK ||
                (st = check_scale(fn, "scale_wt", scale_wt, 1, 1, 1, 1, LCE_E8M0, true)) != LCE_OK)))
        return st;
    const size_t need = lce::linear_blocks_forward_workspace_bytes(n, K, M);
    if (!workspace || workspace_bytes < need)
        return fail(LCE_ERR_INVALID_ARG, "%s: workspace_bytes %zu < minimum %zu", fn, workspace_bytes, need);
    if (!is_aligned(workspace, 256)) return fail(LCE_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", fn);
    const void *ins[4] = {x, weight, bias, residual};
    const void *outs[5] = {out, xt, xt ? scale_xt : nullptr, wt, wt ? scale_wt : nullptr};
    for (int i = 0; i < 5; ++i) {
        for (const void *in : ins)
            if (outs[i] && outs[i] == in && !(i == 0 && in == residual))
                return fail(LCE_ERR_INVALID_ARG, "%s: an output must not be an operand", fn);
        for (int j = 0; j < i; ++j)
            if (outs[i] && outs[i] == outs[j]) return fail(LCE_ERR_INVALID_ARG, "%s: two outputs are the same buffer", fn);
    }
    if ((st = check_residual(fn, residual, ldr, out, ldo, n)) != LCE_OK) return st;
    lce::BlocksForwardArgs a{};
    a.x = x;
    a.weight = weight;
    a.ldx = ldx;
    a.ldw = ldw;
    a.n = n;
    a.K = K;
    a.M = M;
    a.bias = bias;
    a.bias_bf16 = bias_dtype == LCE_BF16;
    a.residual = residual;
    a.ldr = ldr;
    a.out = out;
    a.ldo = ldo;
    a.xt = xt;
    a.wt = wt;
    a.ldxt = ldxt;
    a.ldwt = ldwt;
    a.scale_xt = scale_xt;
    a.scale_wt = scale_wt;
    a.workspace = workspace;
    return hip_status(lce::launch_linear_blocks_forward(a, stream), "lce_linear_blocks_forward launch");
}

size_t lce_linear_blocks_backward_workspace_bytes(int64_t n, int64_t K, int64_t M) {
    if (check_training_sizes("lce_linear_blocks_backward_workspace_bytes", n, K, M) != LCE_OK) return 0;
    return lce::linear_blocks_backward_workspace_bytes(n, K, M);
}

lce_status lce_linear_blocks_backward(const void *grad_out, int64_t ldg, lce_dtype grad_dtype, const void *xt,
                                      int64_t ldxt, const void *scale_xt, int64_t sxt_row, int64_t sxt_col,
                                      const void *wt, int64_t ldwt, const void *scale_wt, int64_t swt_row,
                                      int64_t swt_col, int64_t n, int64_t K, int64_t M, void *grad_x, int64_t ldgx,
                                      void *grad_weight, void *grad_bias, lce_dtype grad_bias_dtype, void *workspace,
                                      size_t workspace_bytes, hipStream_t stream) {
    const char *fn = "lce_linear_blocks_backward";
    lce_status st = check_training_sizes(fn, n, K, M);
    if (st != LCE_OK) return st;
    if (!few_blocks(n, M)) return fail(LCE_ERR_UNSUPPORTED, "%s: 2^24 or more blocks of 128 x 128 in grad_out", fn);
    if (!f32_or_bf16(grad_dtype)) return fail(LCE_ERR_INVALID_ARG, "%s: unknown grad_out dtype %d", fn, (int)grad_dtype);
    if (grad_bias && !f32_or_bf16(grad_bias_dtype))
        return fail(LCE_ERR_INVALID_ARG, "%s: unknown grad_bias dtype %d", fn, (int)grad_bias_dtype);
    const int64_t bn = (n + 127) / 128, bk = (K + 127) / 128, bm = (M + 127) / 128;
    if (n > 0) {
        if ((st = check_matrix(fn, "grad_out", grad_out, ldg, M, grad_dtype, true)) != LCE_OK ||
            (st = check_matrix(fn, "grad_x", grad_x, ldgx, K, LCE_BF16, false)) != LCE_OK)
            return st;
        if (grad_weight && ((st = check_blocked(fn, "xt", xt, ldxt, n)) != LCE_OK ||
                            (st = check_scale(fn, "scale_xt", scale_xt, sxt_row, sxt_col, bk, bn, LCE_E8M0, false)) != LCE_OK))
            return st;
        if (grad_x && ((st = check_blocked(fn, "wt", wt, ldwt, M)) != LCE_OK ||
                       (st = check_scale(fn, "scale_wt", scale_wt, swt_row, swt_col, bk, bm, LCE_E8M0, false)) != LCE_OK))
            return st;
    }
    if (grad_weight && !is_aligned(grad_weight, 2))
        return fail(LCE_ERR_INVALID_ARG, "%s: grad_weight must be 2-byte aligned", fn);
    if (grad_bias && !is_aligned(grad_bias, dtype_bytes(grad_bias_dtype)))
        return fail(LCE_ERR_INVALID_ARG, "%s: grad_bias must be %zu-byte aligned", fn, dtype_bytes(grad_bias_dtype));
    const size_t need = lce::linear_blocks_backward_workspace_bytes(n, K, M);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(LCE_ERR_INVALID_ARG, "%s: workspace_bytes %zu < minimum %zu", fn, workspace_bytes, need);
    if (need > 0 && !is_aligned(workspace, 256))
        return fail(LCE_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", fn);
    const void *ins[5] = {grad_out, xt, scale_xt, wt, scale_wt};
    const void *outs[3] = {grad_x, grad_weight, grad_bias};
    for (int i = 0; i < 3; ++i) {
        for (const void *in : ins)
            if (outs[i] && outs[i] == in) return fail(LCE_ERR_INVALID_ARG, "%s: an output must not be an operand", fn);
        for (int j = 0; j < i; ++j)
            if (outs[i] && outs[i] == outs[j]) return fail(LCE_ERR_INVALID_ARG, "%s: two outputs are the same buffer", fn);
    }
    lce::BlocksGradArgs a{};
    a.grad_out = grad_out;
    a.ldg = ldg;
    a.grad_bf16 = grad_dtype == LCE_BF16;
    a.xt = xt;
    a.ldxt = ldxt;
    a.sxt = {scale_xt, sxt_row, sxt_col, true};
    a.wt = wt;
    a.ldwt = ldwt;
    a.swt = {scale_wt, swt_row, swt_col, true};
    a.n = n;
    a.K = K;
    a.M = M;
    a.grad_x = grad_x;
    a.ldgx = ldgx;
    a.grad_weight = grad_weight;
    a.grad_bias = grad_bias;
    a.grad_bias_bf16 = grad_bias_dtype == LCE_BF16;
    a.workspace = workspace;
    return hip_status(lce::launch_linear_blocks_backward(a, stream), "lce_linear_blocks_backward launch");
}

}  // extern "C"

namespace {

// Sizes of the orthogonalised update: 256 rows of what its products read below 4 GiB, launches below 2^32
// threads.
lce_status check_ortho(const char *fn, int64_t batch, int64_t rows, int64_t cols) {
    if (batch < 0) return fail(LCE_ERR_INVALID_ARG, "%s: batch must be >= 0 (got %lld)", fn, (long long)batch);
    if (rows < 1 || cols < 1)
        return fail(LCE_ERR_INVALID_ARG, "%s: rows and cols must be >= 1 (got %lld, %lld)", fn, (long long)rows, (long long)cols);
    if (rows > (1 << 20) || cols > (1 << 20) || batch > 65535)
        return fail(LCE_ERR_UNSUPPORTED, "%s: rows and cols must be <= 2^20, batch <= 65535", fn);
    // tiles of 64 x 64 in X; up to 64 rows two workgroups of 512 threads each
    const int64_t r = (rows < cols ? rows : cols) / 64 + 1, c = (rows < cols ? cols : rows) / 64 + 1;
    if (r * c >= (int64_t(1) << 22) || batch * r * c >= (int64_t(1) << 22))
        return fail(LCE_ERR_UNSUPPORTED, "%s: 2^22 or more tiles of 64 x 64", fn);
    return LCE_OK;
}

}  // namespace

extern "C" {

size_t lce_orthogonalise_workspace_bytes(int64_t batch, int64_t rows, int64_t cols) {
    if (check_ortho("lce_orthogonalise_workspace_bytes", batch, rows, cols) != LCE_OK) return 0;
    return lce::orthogonalise_workspace_bytes(batch, rows, cols);
}

lce_status lce_orthogonalise(const void *g, int64_t ldg, int64_t g_batch_stride, lce_dtype dtype, int64_t batch,
                             int64_t rows, int64_t cols, int steps, float a, float b, float c, float eps, void *out,
                             int64_t ldo, int64_t out_batch_stride, void *workspace, size_t workspace_bytes,
                             hipStream_t stream) {
    const char *fn = "lce_orthogonalise";
    lce_status st = check_ortho(fn, batch, rows, cols);
    if (st != LCE_OK) return st;
    if (!f32_or_bf16(dtype)) return fail(LCE_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    if (steps < 1 || steps > 100) return fail(LCE_ERR_INVALID_ARG, "%s: steps must be 1 to 100 (got %d)", fn, steps);
    if (!isfinite(a) || !isfinite(b) || !isfinite(c))
        return fail(LCE_ERR_INVALID_ARG, "%s: the coefficients must be finite (got %g, %g, %g)", fn, (double)a, (double)b, (double)c);
    if (!(eps >= 0.0f) || isinf(eps))
        return fail(LCE_ERR_INVALID_ARG, "%s: eps must be finite and >= 0 (got %g)", fn, (double)eps);
    if (!lce::ortho_plan::powers_of(1, steps, a, b, c).fit)
        return fail(LCE_ERR_UNSUPPORTED, "%s: the coefficients (%g, %g, %g) can take singular values past 256 before the last of %d steps",
                    fn, (double)a, (double)b, (double)c, steps);
    if (batch == 0) return ok();
    if ((st = check_matrix(fn, "g", g, ldg, cols, dtype, true)) != LCE_OK ||
        (st = check_matrix(fn, "out", out, ldo, cols, LCE_BF16, true)) != LCE_OK)
        return st;
    if (batch > 1 && g_batch_stride < 0)
        return fail(LCE_ERR_INVALID_ARG, "%s: the batch stride of g must be >= 0", fn);
    const bool apart = out_batch_stride >= (rows - 1) * ldo + cols ||
                       (out_batch_stride >= cols && ldo >= (batch - 1) * out_batch_stride + cols);
    if (batch > 1 && !apart)
        return fail(LCE_ERR_INVALID_ARG, "%s: the batch stride of out (%lld) makes matrices overlap", fn, (long long)out_batch_stride);
    if ((st = check_apart(fn, "out", out, "g", g)) != LCE_OK) return st;
    const size_t need = lce::orthogonalise_workspace_bytes(batch, rows, cols);
    if (!workspace || workspace_bytes < need)
        return fail(LCE_ERR_INVALID_ARG, "%s: workspace_bytes %zu < minimum %zu", fn, workspace_bytes, need);
    if (!is_aligned(workspace, 256))
        return fail(LCE_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", fn);
    lce::OrthoArgs o{};
    o.g = g;
    o.ldg = ldg;
    o.batch_stride = g_batch_stride;
    o.batch = batch;
    o.rows = rows;
    o.cols = cols;
    o.g_bf16 = dtype == LCE_BF16;
    o.out = out;
    o.ldo = ldo;
    o.out_batch_stride = out_batch_stride;
    o.steps = steps;
    o.a = a;
    o.b = b;
    o.c = c;
    o.eps = eps;
    o.workspace = workspace;
    return hip_status(lce::launch_orthogonalise(o, stream), "lce_orthogonalise launch");
}

}  // extern "C"
