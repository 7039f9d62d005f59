// Quantiser into blocks of 128:
//   s_b = the smallest power of two with max |x| <= 448 s_b over block b (1 where that is 0, at least
//         2^-126; NaN where the block holds an infinity or a NaN)
//   q   = e4m3(x / s_b)
// of a matrix and / or of its transpose, each in row blocks (1 x 128) or tiles (128 x 128).
//
// A power of two makes the division exact, so each value is rounded once and the same in any arithmetic,
// and the scale is a byte that the matrix instruction applies by itself.  With max = m 2^E, 1 <= m < 2,
// and 448 = 1.75 2^8 the exponent is E - 8, or E - 7 where m > 1.75: integer work on the bits.  The
// largest magnitude is taken as the integer maximum of the bits without sign, which orders NaN above
// infinity above every number.
//
// A workgroup takes 128 x 128 values, so x is read once whatever is asked for.  A thread holds 8 x 8
// of them: a row's 128 lie in 16 neighbouring lanes, a column's in 16 lanes of four waves, and the eight
// rows of a column make eight neighbouring bytes of the transpose, which goes out through LDS in whole
// 128-byte rows.
//
// Bound by memory: 8192 x 6656 bf16 both ways 41 us, 5.3 TB/s of the 218 MB that it has to move (a copy of
// 1 GiB reaches 5.1); 16384 x 4096 fp32 in tiles both ways 74 to 79 us, 5.1 to 5.4 TB/s.  What got it there
// (8192 x 6656): loads of a whole 8 x 8 without branches (54 -> 41 us with values kept as stored and the
// largest magnitudes taken by pairs; 66 -> 54 with rows that a block ends inside of in one load).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "blocks_internal.h"
#include "ce_device.h"
#include "linear_mfma.h"

namespace lce {
namespace {

using dev::Elt;
using dev::u32x4;

constexpr uint32_t kMinExponent = 1;   // 2^-126

// exponent byte of the scale for the bits of the largest magnitude
__device__ __forceinline__ uint32_t scale_exponent(uint32_t bits) {
    if (bits >= 0x7f800000u) return 255u;   // an infinity or a NaN
    if (bits == 0u) return 127u;
    const uint32_t e = (bits >> 23) + ((bits & 0x7fffffu) > 0x600000u ? 1u : 0u);   // biased exponent of 2^8 s
    return e > 8u + kMinExponent ? e - 8u : kMinExponent;
}
// 1 / s, as x / s = x (1 / s): exact
__device__ __forceinline__ float inverse_scale(uint32_t e) {
    return e == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float((254u - e) << 23);
}
__device__ __forceinline__ void put_scale(const BlockedOut &o, int64_t i, int64_t j, uint32_t e) {
    const int64_t at = i * o.s_row + j * o.s_col;
    if (o.e8m0) static_cast<unsigned char *>(o.scale)[at] = static_cast<unsigned char>(e);
    else static_cast<float *>(o.scale)[at] = e == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(e << 23);
}
// four values as e4m3; the conversion saturates nothing that a scale leaves (|v| <= 448) and keeps NaN
__device__ __forceinline__ uint32_t four(float a, float b, float c, float d) {
    int v = 0;
    v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, v, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
    return static_cast<uint32_t>(v);
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
// the largest of 16 neighbouring lanes
__device__ __forceinline__ uint32_t row16_max(uint32_t m) {
    m = umax(m, static_cast<uint32_t>(dev::dpp_i<dev::kDppXor1>(static_cast<int>(m))));
    m = umax(m, static_cast<uint32_t>(dev::dpp_i<dev::kDppXor2>(static_cast<int>(m))));
    m = umax(m, static_cast<uint32_t>(dev::dpp_i<dev::kDppHalfMirror>(static_cast<int>(m))));
    return umax(m, static_cast<uint32_t>(dev::dpp_i<dev::kDppMirror>(static_cast<int>(m))));
}

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Eight values of a row as they are stored.
template <bool BF16> struct Eight;
template <> struct Eight<true> {
    u32x4 q;
    __device__ __forceinline__ void clear() { q = (u32x4){0u, 0u, 0u, 0u}; }
    __device__ __forceinline__ void load(const void *x, int64_t at) {
        q = *reinterpret_cast<const linear::any16 *>(static_cast<const uint16_t *>(x) + at);
    }
    __device__ __forceinline__ void shift(int up) {
        if (up & 4) q = (u32x4){q.z, q.w, 0u, 0u};
        if (up & 2) q = (u32x4){q.y, q.z, q.w, 0u};
        if (up & 1) q = (u32x4){(q.x >> 16) | (q.y << 16), (q.y >> 16) | (q.z << 16), (q.z >> 16) | (q.w << 16), q.w >> 16};
    }
    __device__ __forceinline__ void set(int e, const void *x, int64_t at) {   // onto zeros
        const uint32_t b = static_cast<const uint16_t *>(x)[at];
        q[e >> 1] |= b << (16 * (e & 1));
    }
    __device__ __forceinline__ float get(int e) const { return Elt<true>::get(q, e); }
    // magnitudes of values 2 w and 2 w + 1
    __device__ __forceinline__ u16x2 pair(int w) const { return __builtin_bit_cast(u16x2, q[w] & 0x7fff7fffu); }
};
template <> struct Eight<false> {
    u32x4 p, s;
    __device__ __forceinline__ void clear() { p = s = (u32x4){0u, 0u, 0u, 0u}; }
    __device__ __forceinline__ void load(const void *x, int64_t at) {
        const linear::any16 *v = reinterpret_cast<const linear::any16 *>(static_cast<const float *>(x) + at);
        p = v[0];
        s = v[1];
    }
    __device__ __forceinline__ void shift(int up) {
        if (up & 4) {
            p = s;
            s = (u32x4){0u, 0u, 0u, 0u};
        }
        if (up & 2) {
            p = (u32x4){p.z, p.w, s.x, s.y};
            s = (u32x4){s.z, s.w, 0u, 0u};
        }
        if (up & 1) {
            p = (u32x4){p.y, p.z, p.w, s.x};
            s = (u32x4){s.y, s.z, s.w, 0u};
        }
    }
    __device__ __forceinline__ void set(int e, const void *x, int64_t at) {
        (e < 4 ? p : s)[e & 3] = __float_as_uint(static_cast<const float *>(x)[at]);
    }
    __device__ __forceinline__ float get(int e) const { return Elt<false>::get(e < 4 ? p : s, e & 3); }
};
// Values c .. c + 7 of N rows, zeros where there are none.  Every lane loads eight values of rows that there are
// and without a branch, so that all loads are under way at once: where c .. c + 7 reach past K, the row's last
// eight, which are then moved up.
template <bool BF16, int N, class Row, class There>
__device__ __forceinline__ void load_rows(const void *x, int64_t c, int64_t K, Row row, There there, Eight<BF16> (&v)[N]) {
    if (K >= 8) {
        const int64_t from = c + 8 <= K ? c : K - 8;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i].load(x, row(i) + from);
        const int up = static_cast<int>(c - from < 8 ? c - from : 8);
        if (up) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                v[i].shift(up);
                if (up >= 8) v[i].clear();
            }
        }
    } else {   // c is 0, or past K
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i].clear();
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (c + e < K) v[i].set(e, x, row(i) + e);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (!there(i)) v[i].clear();
}

__device__ __forceinline__ u16x2 max2(u16x2 a, u16x2 b) { return __builtin_elementwise_max(a, b); }
__device__ __forceinline__ uint32_t widen(uint16_t b) { return static_cast<uint32_t>(b) << 16; }

// Bits of the largest magnitude of eight rows (of eight values each) and of their columns
__device__ __forceinline__ void maxima(const Eight<true> (&v)[8], uint32_t (&rows)[8], uint32_t (&cols)[8]) {
    u16x2 c[4] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        u16x2 r = {};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const u16x2 p = v[i].pair(w);
            r = max2(r, p);
            c[w] = max2(c[w], p);
        }
        rows[i] = umax(widen(r.x), widen(r.y));
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        cols[2 * w] = widen(c[w].x);
        cols[2 * w + 1] = widen(c[w].y);
    }
}
__device__ __forceinline__ void maxima(const Eight<false> (&v)[8], uint32_t (&rows)[8], uint32_t (&cols)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) rows[i] = cols[i] = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t b = __float_as_uint(v[i].get(e)) & 0x7fffffffu;
            rows[i] = umax(rows[i], b);
            cols[e] = umax(cols[e], b);
        }
}
// Keeps the widened values of one use from staying in registers for the next
__device__ __forceinline__ void stay_packed(Eight<true> (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(v[i].q));
}
__device__ __forceinline__ void stay_packed(Eight<false> (&)[8]) {}

// `count` of the bytes of `w`, from the lowest on
__device__ __forceinline__ void put_bytes(unsigned char *o, uint64_t w, int count) {
#pragma unroll 1
    for (int i = 0; i < count; ++i, w >>= 8) o[i] = static_cast<unsigned char>(w);
}
__device__ __forceinline__ void put8(unsigned char *o, uint32_t lo, uint32_t hi, int64_t room) {
    if (room >= 8 && (reinterpret_cast<uintptr_t>(o) & 7) == 0) *reinterpret_cast<uint2 *>(o) = make_uint2(lo, hi);
    else put_bytes(o, lo | static_cast<uint64_t>(hi) << 32, static_cast<int>(room < 8 ? room : 8));
}

// Row blocks alone: 16 lanes a block, wherever it lies, so that few rows keep as many lanes busy as many.
constexpr int kRowBlocks = 4;   // blocks to a lane
template <bool BF16>
__global__ __launch_bounds__(256) void quantize_rows_kernel(QuantizeArgs a, int bk, uint32_t total) {
    const int ch = threadIdx.x & 15;
    const uint32_t first = blockIdx.x * (16u * kRowBlocks) + (threadIdx.x >> 4);
    Eight<BF16> v[kRowBlocks][1];
    uint32_t row[kRowBlocks], b[kRowBlocks];
#pragma unroll
    for (int i = 0; i < kRowBlocks; ++i) {
        const uint32_t at = min(first + i * 16u, total - 1);
        row[i] = at / static_cast<uint32_t>(bk);
        b[i] = at - row[i] * static_cast<uint32_t>(bk);
        load_rows<BF16>(a.x, b[i] * 128ll + ch * 8, a.K, [&](int) { return row[i] * a.ldx; }, [](int) { return true; }, v[i]);
    }
#pragma unroll
    for (int i = 0; i < kRowBlocks; ++i) {
        if (first + i * 16u >= total) break;   // the 16 lanes of a block alike
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = umax(m, __float_as_uint(v[i][0].get(e)) & 0x7fffffffu);
        const uint32_t ex = scale_exponent(row16_max(m));
        if (ch == 0) put_scale(a.q, row[i], b[i], ex);
        const float inv = inverse_scale(ex);
        const int64_t c = b[i] * 128ll + ch * 8;
        if (c < a.K)
            put8(a.q.values + row[i] * a.q.ld + c, four(v[i][0].get(0) * inv, v[i][0].get(1) * inv, v[i][0].get(2) * inv, v[i][0].get(3) * inv),
                 four(v[i][0].get(4) * inv, v[i][0].get(5) * inv, v[i][0].get(6) * inv, v[i][0].get(7) * inv), a.K - c);
    }
}

// Up to two matrices in a launch
struct QuantizeJobs {
    QuantizeArgs job[2];
    int tiles_c[2];
    unsigned first_tiles;   // of job 0
};
template <bool BF16>
__global__ __launch_bounds__(256) void quantize_kernel(QuantizeJobs jobs) {
    __shared__ __attribute__((aligned(16))) unsigned char flat[128 * 128];   // the transpose: 16-byte chunk c of row r at c ^ (r / 8 mod 8)
    __shared__ uint32_t col_max[4][128];
    __shared__ float col_sum[4][128];
    __shared__ uint32_t wave_max[4];
    const int which = blockIdx.x < jobs.first_tiles ? 0 : 1;
    const QuantizeArgs &a = jobs.job[which];
    const int tile = static_cast<int>(blockIdx.x - (which ? jobs.first_tiles : 0u)), tiles_c = jobs.tiles_c[which];
    const int br = tile / tiles_c, bc = tile - br * tiles_c;
    const int64_t r0 = br * 128ll, c0 = bc * 128ll;
    const int t = threadIdx.x, ch = t & 15, g = t >> 4, lane = t & 63, wave = t >> 6;
    const int64_t gr = r0 + g * 8, gc = c0 + ch * 8;
    Eight<BF16> v[8];   // rows gr .. gr + 7, columns gc .. gc + 7
    load_rows<BF16>(a.x, gc, a.K, [&](int i) { return (gr + i < a.n ? gr + i : a.n - 1) * a.ldx; },
                    [&](int i) { return gr + i < a.n; }, v);
    uint32_t rmax[8], cmax[8], all = 0;
    maxima(v, rmax, cmax);
    const bool want_tile = (a.q.values && a.q.tile) || (a.qt.values && a.qt.tile);
    if (want_tile) {
#pragma unroll
        for (int i = 0; i < 8; ++i) all = umax(all, rmax[i]);
        all = row16_max(all);
        all = umax(all, static_cast<uint32_t>(__shfl_xor(static_cast<int>(all), 16)));
        all = umax(all, static_cast<uint32_t>(__shfl_xor(static_cast<int>(all), 32)));
        if (lane == 0) wave_max[wave] = all;
    }
    if (a.qt.values && !a.qt.tile) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint32_t c = cmax[e];
            c = umax(c, static_cast<uint32_t>(__shfl_xor(static_cast<int>(c), 16)));
            c = umax(c, static_cast<uint32_t>(__shfl_xor(static_cast<int>(c), 32)));
            if (lane < 16) col_max[wave][ch * 8 + e] = c;
        }
    }
    if (a.part) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float c = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) c += v[i].get(e);
            c += __shfl_xor(c, 16);
            c += __shfl_xor(c, 32);
            if (lane < 16) col_sum[wave][ch * 8 + e] = c;
        }
    }
    stay_packed(v);
    __syncthreads();
    uint32_t tile_e = 0;
    if (want_tile) {
        all = umax(umax(wave_max[0], wave_max[1]), umax(wave_max[2], wave_max[3]));
        tile_e = scale_exponent(all);
        if (t == 0 && a.q.values && a.q.tile) put_scale(a.q, br, bc, tile_e);
        if (t == 0 && a.qt.values && a.qt.tile) put_scale(a.qt, bc, br, tile_e);
    }
    if (a.part && t < 128 && c0 + t < a.K)
        a.part[br * a.K + c0 + t] = (col_sum[0][t] + col_sum[1][t]) + (col_sum[2][t] + col_sum[3][t]);
    if (a.q.values) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t e = tile_e;
            if (!a.q.tile) {
                e = scale_exponent(row16_max(rmax[i]));
                if (ch == 0 && gr + i < a.n) put_scale(a.q, gr + i, bc, e);
            }
            const float inv = inverse_scale(e);
            const uint32_t lo = four(v[i].get(0) * inv, v[i].get(1) * inv, v[i].get(2) * inv, v[i].get(3) * inv);
            const uint32_t hi = four(v[i].get(4) * inv, v[i].get(5) * inv, v[i].get(6) * inv, v[i].get(7) * inv);
            if (gr + i < a.n && gc < a.K) put8(a.q.values + (gr + i) * a.q.ld + gc, lo, hi, a.K - gc);
        }
    }
    if (!a.qt.values) return;
    stay_packed(v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int c = ch * 8 + e;
        uint32_t ex = tile_e;
        if (!a.qt.tile) {
            ex = scale_exponent(umax(umax(col_max[0][c], col_max[1][c]), umax(col_max[2][c], col_max[3][c])));
            if (g == 0 && c0 + c < a.K) put_scale(a.qt, c0 + c, br, ex);
        }
        const float inv = inverse_scale(ex);
        const uint2 w = make_uint2(four(v[0].get(e) * inv, v[1].get(e) * inv, v[2].get(e) * inv, v[3].get(e) * inv),
                                   four(v[4].get(e) * inv, v[5].get(e) * inv, v[6].get(e) * inv, v[7].get(e) * inv));
        *reinterpret_cast<uint2 *>(flat + c * 128 + (((g >> 1) ^ (ch & 7)) * 16) + (g & 1) * 8) = w;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const int idx = t + h * 256, c = idx >> 3, chunk = idx & 7;
        const int64_t row = c0 + c, col = r0 + chunk * 16;
        if (row >= a.K || col >= a.n) continue;
        const u32x4 q = *reinterpret_cast<const u32x4 *>(flat + c * 128 + ((chunk ^ ((c >> 3) & 7)) * 16));
        unsigned char *o = a.qt.values + row * a.qt.ld + col;
        const int64_t room = a.n - col;
        if (room >= 16 && (reinterpret_cast<uintptr_t>(o) & 15) == 0) {
            *reinterpret_cast<u32x4 *>(o) = q;
        } else {
            put_bytes(o, q.x | static_cast<uint64_t>(q.y) << 32, static_cast<int>(room < 8 ? room : 8));
            put_bytes(o + 8, q.z | static_cast<uint64_t>(q.w) << 32, static_cast<int>(room < 16 ? room - 8 : 8));
        }
    }
}

int64_t tiles_of(const QuantizeArgs &a) { return ((a.n + 127) / 128) * ((a.K + 127) / 128); }

}  // namespace

hipError_t launch_quantize_blocks(const QuantizeArgs &a, bool is_bf16, hipStream_t st) {
    if (a.n <= 0 || a.K <= 0) return hipSuccess;
    const int64_t tiles = tiles_of(a), bk = (a.K + 127) / 128, blocks = a.n * bk;
    if (tiles >= (int64_t(1) << 24)) return hipErrorInvalidValue;
    // up to 64 rows they have fewer lanes without work: 16 x 6656 bf16 4.4 us, with tiles of 128 rows 7.6
    if (a.q.values && !a.q.tile && !a.qt.values && !a.part && a.n <= 64 && blocks < (int64_t(1) << 31)) {
        const dim3 grid(static_cast<unsigned>((blocks + 16 * kRowBlocks - 1) / (16 * kRowBlocks)));
        if (is_bf16) hipLaunchKernelGGL((quantize_rows_kernel<true>), grid, dim3(256), 0, st, a, static_cast<int>(bk), static_cast<uint32_t>(blocks));
        else hipLaunchKernelGGL((quantize_rows_kernel<false>), grid, dim3(256), 0, st, a, static_cast<int>(bk), static_cast<uint32_t>(blocks));
        return hipGetLastError();
    }
    QuantizeJobs jobs{};
    jobs.job[0] = a;
    jobs.tiles_c[0] = static_cast<int>(bk);
    jobs.first_tiles = static_cast<unsigned>(tiles);
    if (is_bf16) hipLaunchKernelGGL((quantize_kernel<true>), dim3(jobs.first_tiles), dim3(256), 0, st, jobs);
    else hipLaunchKernelGGL((quantize_kernel<false>), dim3(jobs.first_tiles), dim3(256), 0, st, jobs);
    return hipGetLastError();
}

hipError_t launch_quantize_pair(const QuantizeArgs &a, const QuantizeArgs &b, hipStream_t st) {
    const int64_t first = tiles_of(a), second = tiles_of(b);
    if (first + second >= (int64_t(1) << 24)) return hipErrorInvalidValue;
    if (first + second == 0) return hipSuccess;
    QuantizeJobs jobs{};
    jobs.job[0] = a;
    jobs.job[1] = b;
    jobs.tiles_c[0] = static_cast<int>((a.K + 127) / 128);
    jobs.tiles_c[1] = static_cast<int>((b.K + 127) / 128);
    jobs.first_tiles = static_cast<unsigned>(first);
    hipLaunchKernelGGL((quantize_kernel<true>), dim3(static_cast<unsigned>(first + second)), dim3(256), 0, st, jobs);
    return hipGetLastError();
}

}  // namespace lce
