// Rules on logits before a token is drawn, for gfx950: softcap, penalties for
// tokens already seen, biases, temperature and grammar masks, in one pass.
//
// For row i, column j, with c = how often j was generated (history past the
// prompt) and seen = j in the history at all:
//
//   z = softcap > 0 ? T tanh(x / T) : x
//   z = seen ? (z > 0 ? z / repetition_i : z repetition_i) : z
//   z = z - frequency_i c - presence_i [c > 0]
//   z = z + bias of j (its last entry in row i's list)
//   z = temperature_i > 0 ? z / temperature_i : z
//   out = allowed(mask row of i, j) ? z : mask_value
//
// Bound by memory: each logit is read once and written once.  A workgroup takes
// a slice of a row's columns and keeps one LDS word per column of it: bit 31 says
// that the prompt holds the token, the low bits count it among the generated ones
// (integer atomics, so the order of the history does not change the result), and
// with biases a second word holds the last entry's index plus one.  So the
// history is read once per slice, from L2 after the first, no table of counts over
// the vocabulary exists in memory, and nothing is kept between calls.  The
// slice's logits are requested before the history is scanned and wait in
// registers meanwhile.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ce_device.h"
#include "head_internal.h"

namespace lce {
namespace {

using dev::Elt;
using dev::u32x4;

constexpr int kThreads = 256;
constexpr int kVecs = 4;                        // 16-byte vectors of logits per thread
constexpr int kSliceVecs = kThreads * kVecs;    // ... per workgroup
constexpr uint32_t kPrompt = 0x80000000u;

// T tanh(u), u = x / T: an odd polynomial near zero (its next term is below 2^-28
// of u at 0.25), else (1 - t) / (1 + t) with t = e^{-2 |u|} <= 1.
__device__ __forceinline__ float softcapped(float x, float T, float inv_t) {
    const float u = x * inv_t, au = fabsf(u), u2 = u * u;
    const float t = dev::exp2_fast(au * (-2.0f * dev::kLog2e));
    const float big = copysignf((1.0f - t) * dev::rcp_fast(1.0f + t), u);
    const float poly =
        u * fmaf(u2, fmaf(u2, fmaf(u2, fmaf(u2, 62.0f / 2835.0f, -17.0f / 315.0f), 2.0f / 15.0f), -1.0f / 3.0f), 1.0f);
    return T * (au < 0.25f ? poly : big);
}

template <bool BF16, typename Id, bool HIST, bool BIAS>
__global__ __launch_bounds__(kThreads) void logits_process_kernel(RulesArgs a, unsigned slices) {
    constexpr int E = Elt<BF16>::E, BYTES = Elt<BF16>::bytes;
    constexpr int COLS = kSliceVecs * E;
    __shared__ __attribute__((aligned(16))) uint32_t counts[HIST ? COLS : 4];
    __shared__ __attribute__((aligned(16))) uint32_t entries[BIAS ? COLS : 4];
    // workgroups are dealt round robin over the 8 XCDs: a row's slices go to one XCD, whose L2
    // then holds its history
    const unsigned b = blockIdx.x;
    const int64_t row = static_cast<int64_t>(b / 8 / slices) * 8 + (b & 7);
    if (row >= a.n) return;
    const int64_t slice = (b / 8) % slices;
    const char *xrow = static_cast<const char *>(a.logits) + row * a.ldx * BYTES;
    char *orow = static_cast<char *>(a.out) + row * a.ldo * BYTES;
    // the row is taken in 16-byte windows of the address space: `lead` elements of the first lie before it
    const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(xrow) & 15) / BYTES);
    const bool vec_out = (reinterpret_cast<uintptr_t>(orow) & 15) / BYTES == static_cast<uintptr_t>(lead);
    const int64_t base = slice * COLS - lead;   // column of the slice's first element
    const int V = static_cast<int>(a.V);

    float x[kVecs][E];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        const int64_t c = base + (k * kThreads + static_cast<int>(threadIdx.x)) * E;
        if (c >= 0 && c + E <= V) {
            const u32x4 q = *reinterpret_cast<const u32x4 *>(xrow + c * BYTES);
#pragma unroll
            for (int e = 0; e < E; ++e) x[k][e] = Elt<BF16>::get(q, e);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) x[k][e] = (c + e >= 0 && c + e < V) ? Elt<BF16>::load_one(xrow, c + e) : 0.0f;
        }
    }

    int64_t len = 0;
    if constexpr (HIST) {
        len = a.L;
        if (a.history_lens) {
            const int64_t l = a.history_lens[row];
            len = l < 0 ? 0 : (l < a.L ? l : a.L);
        }
    }
    if constexpr (HIST || BIAS) {
        const u32x4 zero = {0u, 0u, 0u, 0u};
        for (int i = threadIdx.x; i < COLS / 4; i += kThreads) {
            if constexpr (HIST) reinterpret_cast<u32x4 *>(counts)[i] = zero;
            if constexpr (BIAS) reinterpret_cast<u32x4 *>(entries)[i] = zero;
        }
        __syncthreads();
        if constexpr (HIST) {
            const Id *h = static_cast<const Id *>(a.history) + row * a.ldh;
            const int64_t prompt = a.prompt_lens ? a.prompt_lens[row] : 0;
            for (int64_t i0 = threadIdx.x; i0 < len; i0 += 4 * kThreads) {
                Id id[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) id[u] = i0 + u * kThreads < len ? h[i0 + u * kThreads] : static_cast<Id>(-1);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (id[u] < 0 || id[u] >= static_cast<Id>(V)) continue;   // padding
                    const int64_t at = static_cast<int64_t>(id[u]) - base;
                    if (at < 0 || at >= COLS) continue;
                    if (i0 + u * kThreads < prompt) atomicOr(&counts[at], kPrompt);
                    else atomicAdd(&counts[at], 1u);
                }
            }
        }
        if constexpr (BIAS) {
            const Id *ids = static_cast<const Id *>(a.bias_ids) + row * a.ldbi;
            for (int64_t i = threadIdx.x; i < a.B; i += kThreads) {
                const Id id = ids[i];
                if (id < 0 || id >= static_cast<Id>(V)) continue;
                const int64_t at = static_cast<int64_t>(id) - base;
                if (at >= 0 && at < COLS) atomicMax(&entries[at], static_cast<uint32_t>(i + 1));
            }
        }
        __syncthreads();
    }

    const float rep = a.repetition ? a.repetition[row] : 1.0f;
    const float pres = a.presence ? a.presence[row] : 0.0f;
    const float freq = a.frequency ? a.frequency[row] : 0.0f;
    const float temp = a.temperature ? a.temperature[row] : 0.0f;
    const float inv_temp = temp > 0.0f ? 1.0f / temp : 1.0f;
    const float cap = a.softcap, inv_cap = cap > 0.0f ? 1.0f / cap : 0.0f;
    const float *bias = BIAS ? a.bias_values + row * a.ldbv : nullptr;
    const uint32_t *words = nullptr;
    if (a.allowed) {
        const int64_t r = a.mask_rows ? a.mask_rows[row] : row;
        if (r >= 0 && r < a.R) words = a.allowed + r * a.ldm;
    }
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        const int local = (k * kThreads + static_cast<int>(threadIdx.x)) * E;
        const int64_t c = base + local;
        if (c >= V) continue;
        uint32_t bits = ~0u;   // bit e: column c + e is allowed
        if (words) {
            // columns c .. c + E - 1 lie in one word or two; those before the row or past V do not matter
            const int64_t c0 = c < 0 ? 0 : c;
            const int64_t c1 = c + E - 1 < V ? c + E - 1 : V - 1;
            const uint64_t lo = words[c0 >> 5], hi = words[c1 >> 5];
            bits = static_cast<uint32_t>(((hi << 32) | lo) >> (c0 & 31));
            if ((c0 >> 5) == (c1 >> 5)) bits = static_cast<uint32_t>(lo >> (c0 & 31));
            if (c < 0) bits <<= -c;
        }
        float o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            float z = x[k][e];
            if (cap > 0.0f) z = softcapped(z, cap, inv_cap);
            if constexpr (HIST) {
                const uint32_t n = counts[local + e];
                if (n) {
                    z = z > 0.0f ? z / rep : z * rep;
                    const uint32_t made = n & ~kPrompt;
                    if (made) z = z - freq * static_cast<float>(made) - pres;
                }
            }
            if constexpr (BIAS) {
                const uint32_t n = entries[local + e];
                if (n) z += bias[n - 1];
            }
            z *= inv_temp;
            o[e] = (bits >> e) & 1 ? z : a.mask_value;
        }
        if (vec_out && c >= 0 && c + E <= V) {
            *reinterpret_cast<u32x4 *>(orow + c * BYTES) = Elt<BF16>::pack(o);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (c + e >= 0 && c + e < V) Elt<BF16>::store_one(orow, c + e, o[e]);
        }
    }
}

template <bool BF16, typename Id, bool HIST, bool BIAS>
hipError_t launch(const RulesArgs &a, hipStream_t st) {
    constexpr int COLS = kSliceVecs * Elt<BF16>::E;
    // a row that starts inside a 16-byte window covers up to E - 1 elements more
    const int64_t slices = (a.V + Elt<BF16>::E - 1 + COLS - 1) / COLS;
    // a launch has fewer than 2^32 threads
    const int64_t rows = ((int64_t(1) << 23) / slices) / 8 * 8;
    for (int64_t r = 0; r < a.n; r += rows) {
        RulesArgs b = a;
        b.n = a.n - r < rows ? a.n - r : rows;
        const int64_t es = Elt<BF16>::bytes, is = sizeof(Id);
        b.logits = static_cast<const char *>(a.logits) + r * a.ldx * es;
        b.out = static_cast<char *>(a.out) + r * a.ldo * es;
        auto skip = [&](auto *p, int64_t n) { return p ? p + n : p; };
        b.history = skip(static_cast<const char *>(a.history), r * a.ldh * is);
        b.history_lens = skip(a.history_lens, r);
        b.prompt_lens = skip(a.prompt_lens, r);
        b.bias_ids = skip(static_cast<const char *>(a.bias_ids), r * a.ldbi * is);
        b.bias_values = skip(a.bias_values, r * a.ldbv);
        b.repetition = skip(a.repetition, r);
        b.presence = skip(a.presence, r);
        b.frequency = skip(a.frequency, r);
        b.temperature = skip(a.temperature, r);
        if (a.mask_rows) {
            b.mask_rows = a.mask_rows + r;
        } else if (a.allowed) {   // row i uses mask row i
            b.allowed = a.allowed + r * a.ldm;
            b.R = a.R - r;
        }
        const unsigned grid = static_cast<unsigned>((b.n + 7) / 8 * 8 * slices);
        hipLaunchKernelGGL((logits_process_kernel<BF16, Id, HIST, BIAS>), dim3(grid), dim3(kThreads), 0, st, b,
                           static_cast<unsigned>(slices));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <bool BF16, typename Id>
hipError_t pick(const RulesArgs &a, hipStream_t st) {
    if (a.history) return a.bias_ids ? launch<BF16, Id, true, true>(a, st) : launch<BF16, Id, true, false>(a, st);
    return a.bias_ids ? launch<BF16, Id, false, true>(a, st) : launch<BF16, Id, false, false>(a, st);
}

}  // namespace

hipError_t launch_logits_process(const RulesArgs &a, bool is_bf16, hipStream_t st) {
    if (a.n == 0) return hipSuccess;
    if (is_bf16) return a.id64 ? pick<true, int64_t>(a, st) : pick<true, int32_t>(a, st);
    return a.id64 ? pick<false, int64_t>(a, st) : pick<false, int32_t>(a, st);
}

}  // namespace lce
