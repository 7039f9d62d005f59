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
// a slice of a row's columns and keeps one LDS word per column of it.  First the
// lists are scanned and the word counts: bit 31 says that the prompt holds the
// token, the bits below count it among the generated ones (integer atomics, so the
// order of the history does not change the result); a bias list leaves its last
// entry's index plus one for the column.  Whoever touches a column first puts it
// on the slice's list.  Then the listed columns, few, are worked out one per lane
// and their words replaced by the result's bits; the sweep over all columns only
// selects between a word and the common case.  (Working the penalties out inside
// the sweep ran a division in half of its steps for a wave's one or two listed
// columns: 114 us where this took 67, 256 x 131072 bf16 with every rule, before the
// steps below brought it to 38.)  Without lists the same logits take 26 us, 5.2 TB/s,
// what a copy takes; with them a workgroup's chain of dependent loads and barriers
// (history, counts, listed columns, sweep) is what remains.  The history is read once per slice, from L2 after the first, no table of counts over
// the vocabulary exists in memory, and nothing is kept between calls.  The slice's
// logits are requested before the history is scanned and wait in registers.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ce_device.h"
#include "head_internal.h"

namespace lce {
namespace {

using dev::Elt;
using dev::u32x4;

// 16 bytes at any address (gfx950 stores them in one instruction): the output's rows need not start
// where the logits' do
typedef uint32_t any16 __attribute__((ext_vector_type(4), aligned(2)));

constexpr int kThreads = 512;
constexpr uint32_t kPrompt = 0x80000000u;
constexpr int kAhead = 4;   // history ids per thread requested at once

// How biases are kept: none; the last entry's index plus one in the low 16 bits of the column's word,
// the count above it (histories below 2^15 tokens, lists below 2^16 entries); or in a word of its own.
// With a word of its own everywhere, half as many columns fit a workgroup: 256 x 131072 bf16 with every
// rule took 67 us where the packed word takes 38.
enum BiasMode { NO_BIAS = 0, PACKED = 1, OWN_WORD = 2 };
constexpr int64_t kPackedL = 1 << 15, kPackedB = (1 << 16) - 1;
// Columns a slice lists; with more (a long text without repetition) the sparse step looks at every
// column's word instead: 33 x 50257 with 16384 distinct tokens 18 us, with 8192 10 us.
constexpr uint32_t kListed = 2048;

// 16-byte vectors of logits per thread: 8192 columns per workgroup, half with words for the biases
// (four workgroups per CU either way).
template <bool BF16, int BIAS>
constexpr int vecs_of() { return 8192 / (kThreads * Elt<BF16>::E) / (BIAS == OWN_WORD ? 2 : 1); }

// T tanh(x / T), with v = x / T.  Near zero an odd polynomial in v, else (1 - t) / (1 + t) with
// t = e^{-2 |v|} <= 1, whose difference loses 2^-24 / |v| of itself there.  fp32 logits need all of fp32:
// five terms up to |v| = 1 / 4 (the next is below 2^-28 of x); bf16 ones are rounded 2^15 times coarser: two
// terms up to 1 / 64 (2^-27), the quotient exact to 2^-18 beyond.  Nothing but v overflows, whatever T is, and
// then t is 0.  (1 / temperature is a factor of its own: in T it overflowed for small temperatures, which
// made NaN of finite logits.)
struct Softcap {
    float T, u;
    __device__ __forceinline__ explicit Softcap(float cap) : T(cap), u(fminf(1.0f / cap, FLT_MAX)) {}
};
template <bool BF16>
__device__ __forceinline__ float softcapped(float x, const Softcap &s) {
    const float v = x * s.u, v2 = v * v;
    const float t = dev::exp2_fast(fabsf(v) * (-2.0f * dev::kLog2e));
    const float big = copysignf(fmaf(-s.T, t, s.T) * dev::rcp_fast(1.0f + t), x);
    if constexpr (BF16) {
        return fabsf(v) < 0.015625f ? x * fmaf(v2, -1.0f / 3.0f, 1.0f) : big;
    } else {
        const float p =
            fmaf(v2, fmaf(v2, fmaf(v2, fmaf(v2, 62.0f / 2835.0f, -17.0f / 315.0f), 2.0f / 15.0f), -1.0f / 3.0f), 1.0f);
        return fabsf(v) < 0.25f ? x * p : big;
    }
}

template <bool BF16, typename Id, bool HIST, int BIAS>
__global__ __launch_bounds__(kThreads) void logits_process_kernel(RulesArgs a, unsigned slices) {
    constexpr int E = Elt<BF16>::E, BYTES = Elt<BF16>::bytes, VECS = vecs_of<BF16, BIAS>();
    constexpr int COLS = kThreads * VECS * E;
    constexpr bool SPARSE = HIST || BIAS;
    constexpr int SHIFT = BIAS == PACKED ? 16 : 0;   // where the count starts
    __shared__ __attribute__((aligned(16))) uint32_t table[SPARSE ? COLS : 4];
    __shared__ __attribute__((aligned(16))) uint32_t own[BIAS == OWN_WORD ? COLS : 4];
    __shared__ uint16_t list[SPARSE ? kListed : 4];
    __shared__ uint32_t listed;
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
    const int V = static_cast<int>(a.V);
    const int base = static_cast<int>(slice * COLS) - lead;   // column of the slice's first element
    if (base >= V) return;
    const int tid = threadIdx.x;

    // Everything whose address is known goes out first: a workgroup's time is the chain of its
    // dependent loads, not its arithmetic.
    const Id *h = HIST ? static_cast<const Id *>(a.history) + row * a.ldh : nullptr;
    const Id *bids = BIAS ? static_cast<const Id *>(a.bias_ids) + row * a.ldbi : nullptr;
    Id ahead[kAhead], bid = static_cast<Id>(-1);
    if constexpr (BIAS) {
        if (tid < a.B) bid = bids[tid];
    }
    if constexpr (HIST) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            ahead[u] = tid + u * kThreads < a.L ? h[tid + u * kThreads] : static_cast<Id>(-1);
    }
    u32x4 x[VECS];
#pragma unroll
    for (int k = 0; k < VECS; ++k) {
        const int c = base + (k * kThreads + tid) * E;
        x[k] = (u32x4){0u, 0u, 0u, 0u};
        if (c >= 0 && c + E <= V) {
            x[k] = *reinterpret_cast<const u32x4 *>(xrow + static_cast<int64_t>(c) * BYTES);
        } else if (c < V) {
            float v[E];
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = (c + e >= 0 && c + e < V) ? Elt<BF16>::load_one(xrow, c + e) : 0.0f;
            x[k] = Elt<BF16>::pack(v);
        }
    }
    const float temp = a.temperature ? a.temperature[row] : 0.0f;
    const float cap = a.softcap;
    const float rep = a.repetition ? a.repetition[row] : 1.0f;
    const float pres = a.presence ? a.presence[row] : 0.0f;
    const float freq = a.frequency ? a.frequency[row] : 0.0f;
    const uint32_t *words = nullptr;
    if (a.allowed) {
        const int64_t r = a.mask_rows ? a.mask_rows[row] : row;
        if (r >= 0 && r < a.R) words = a.allowed + r * a.ldm;
    }
    // A factor in place of a division, ten instructions a logit: one rounding more (2^-24 of a value that bf16
    // rounds to 2^-9; fp32 logits with every rule are off by 4e-8 on the whole, 2.5e-8 with divisions).
    const float inv_temp = temp > 0.0f ? fminf(1.0f / temp, FLT_MAX) : 1.0f;   // finite, so that 0 stays 0
    // mask bits of columns c .. c + E - 1: they lie in one word or two (those before the row or past V do
    // not matter)
    uint32_t lo[VECS], hi[VECS];
#pragma unroll
    for (int k = 0; k < VECS; ++k) {
        const int c = base + (k * kThreads + tid) * E;
        lo[k] = hi[k] = 0;
        if (words && c < V) {
            lo[k] = words[(c < 0 ? 0 : c) >> 5];
            hi[k] = words[(c + E - 1 < V ? c + E - 1 : V - 1) >> 5];
        }
    }

    if constexpr (SPARSE) {
        const u32x4 zero = {0u, 0u, 0u, 0u};
        for (int i = tid; i < COLS / 4; i += kThreads) {
            reinterpret_cast<u32x4 *>(table)[i] = zero;
            if constexpr (BIAS == OWN_WORD) reinterpret_cast<u32x4 *>(own)[i] = zero;
        }
        if (tid == 0) listed = 0;
        __syncthreads();
        auto push = [&](int at) {
            const uint32_t i = atomicAdd(&listed, 1u);
            if (i < kListed) list[i] = static_cast<uint16_t>(at);
        };
        auto column = [&](Id id) {   // of the slice, or -1: padding or another slice's
            if (id < 0 || id >= static_cast<Id>(V)) return -1;
            const int at = static_cast<int>(id) - base;
            return at < COLS ? at : -1;   // below the slice: negative already
        };
        if constexpr (BIAS) {
            uint32_t *entries = BIAS == PACKED ? table : own;
            for (int64_t i = tid; i < a.B; i += kThreads) {
                const int at = column(i == tid ? bid : bids[i]);
                if (at < 0) continue;
                const uint32_t old = atomicMax(&entries[at], static_cast<uint32_t>(i + 1));
                if (old == 0) push(at);
            }
            // a packed word is an entry until here, then counts: the order of the two must not mix; with
            // words of their own a listed column must not be listed again
            if constexpr (HIST) __syncthreads();
        }
        if constexpr (HIST) {
            int64_t len = a.L;
            if (a.history_lens) {
                const int64_t l = a.history_lens[row];
                len = l < 0 ? 0 : (l < a.L ? l : a.L);
            }
            const int64_t prompt = a.prompt_lens ? a.prompt_lens[row] : 0;
            for (int64_t i0 = tid; i0 < len; i0 += kAhead * kThreads) {
                if (i0 != tid) {
#pragma unroll
                    for (int u = 0; u < kAhead; ++u)
                        ahead[u] = i0 + u * kThreads < len ? h[i0 + u * kThreads] : static_cast<Id>(-1);
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    if (i0 + u * kThreads >= len) continue;
                    const int at = column(ahead[u]);
                    if (at < 0) continue;
                    const uint32_t old =
                        i0 + u * kThreads < prompt ? atomicOr(&table[at], kPrompt) : atomicAdd(&table[at], 1u << SHIFT);
                    if (old == 0 && (BIAS != OWN_WORD || own[at] == 0)) push(at);
                }
            }
        }
        __syncthreads();
        // the listed columns, one per lane
        const bool all = listed > kListed;
        const int n = all ? COLS : static_cast<int>(listed);
        for (int i = tid; i < n; i += kThreads) {
            const int at = all ? i : list[i];
            const uint32_t word = table[at];
            if (all && word == 0 && (BIAS != OWN_WORD || own[at] == 0)) continue;
            float z = Elt<BF16>::load_one(xrow, base + at);
            uint32_t entry = 0;
            if constexpr (BIAS == PACKED) entry = word & 0xffffu;
            else if constexpr (BIAS == OWN_WORD) entry = own[at];
            float bias = 0.0f;
            if constexpr (BIAS) {
                if (entry) bias = a.bias_values[row * a.ldbv + entry - 1];
            }
            if (cap > 0.0f) z = softcapped<BF16>(z, Softcap(cap));
            if constexpr (HIST) {
                const uint32_t made = (word & ~kPrompt) >> SHIFT;
                if (made | (word & kPrompt)) z = z > 0.0f ? z / rep : z * rep;
                if (made) z = z - freq * static_cast<float>(made) - pres;
            }
            if constexpr (BIAS) {
                if (entry) z += bias;
            }
            const uint32_t bits = __float_as_uint(z * inv_temp);
            table[at] = bits ? bits : 0x80000000u;   // 0 says that nothing is listed: -0 for 0
        }
        __syncthreads();
    }

    const uint32_t hidden = __float_as_uint(a.mask_value);
    const Softcap capped(cap > 0.0f ? cap : 1.0f);
#pragma unroll
    for (int k = 0; k < VECS; ++k) {
        const int local = (k * kThreads + tid) * E;
        const int c = base + local;
        if (c >= V) continue;
        float o[E];
        if (cap > 0.0f) {
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = softcapped<BF16>(Elt<BF16>::get(x[k], e), capped) * inv_temp;
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = Elt<BF16>::get(x[k], e) * inv_temp;
        }
        if constexpr (SPARSE) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const uint32_t w = table[local + e];
                o[e] = w ? __uint_as_float(w) : o[e];
            }
        }
        if (words) {
            const int c0 = c < 0 ? 0 : c, c1 = c + E - 1 < V ? c + E - 1 : V - 1;
            uint32_t bits = static_cast<uint32_t>(((static_cast<uint64_t>(hi[k]) << 32) | lo[k]) >> (c0 & 31));
            if ((c0 >> 5) == (c1 >> 5)) bits = lo[k] >> (c0 & 31);   // bit e: column c + e is allowed
            if (c < 0) bits <<= -c;
#pragma unroll
            for (int e = 0; e < E; ++e) {   // all ones or all zeros from bit e, then one bit-field select
                const uint32_t keep = static_cast<uint32_t>(__builtin_amdgcn_sbfe(static_cast<int>(bits), e, 1));
                o[e] = __uint_as_float((keep & __float_as_uint(o[e])) | (~keep & hidden));
            }
        }
        if (c >= 0 && c + E <= V) {
            *reinterpret_cast<any16 *>(orow + static_cast<int64_t>(c) * BYTES) = Elt<BF16>::pack(o);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (c + e >= 0 && c + e < V) Elt<BF16>::store_one(orow, c + e, o[e]);
        }
    }
}

template <bool BF16, typename Id, bool HIST, int BIAS>
hipError_t launch(const RulesArgs &a, hipStream_t st) {
    constexpr int COLS = kThreads * vecs_of<BF16, BIAS>() * Elt<BF16>::E;
    // a row that starts inside a 16-byte window covers up to E - 1 elements more
    const bool aligned = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && a.ldx * Elt<BF16>::bytes % 16 == 0;
    const int64_t slices = (a.V + (aligned ? 0 : Elt<BF16>::E - 1) + COLS - 1) / COLS;
    // a launch has fewer than 2^32 threads
    const int64_t rows = ((int64_t(1) << 22) / slices) / 8 * 8;   // slices <= 2^19
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
    if (!a.bias_ids) return a.history ? launch<BF16, Id, true, NO_BIAS>(a, st) : launch<BF16, Id, false, NO_BIAS>(a, st);
    if (!a.history) return a.B <= kPackedB ? launch<BF16, Id, false, PACKED>(a, st) : launch<BF16, Id, false, OWN_WORD>(a, st);
    return a.L < kPackedL && a.B <= kPackedB ? launch<BF16, Id, true, PACKED>(a, st) : launch<BF16, Id, true, OWN_WORD>(a, st);
}

}  // namespace

hipError_t launch_logits_process(const RulesArgs &a, bool is_bf16, hipStream_t st) {
    if (a.n == 0) return hipSuccess;
    if (is_bf16) return a.id64 ? pick<true, int64_t>(a, st) : pick<true, int32_t>(a, st);
    return a.id64 ? pick<false, int64_t>(a, st) : pick<false, int32_t>(a, st);
}

}  // namespace lce
