// Device helpers of the paged key-value cache's kernels.
#pragma once

#include "common.h"
#include "kv.h"

namespace w4 {

// Page that holds tokens [16 i, 16 i + 16) of a table row, or -1: an entry
// outside [0, pages) or beyond the row is no page.
__device__ __forceinline__ int kv_page(const KvView &c, const int32_t *row, int64_t token) {
    const int64_t j = token >> c.shift;
    if (j >= c.W) return -1;
    const int p = row[j];
    return (uint32_t)p < (uint32_t)c.pages ? p : -1;
}

// The sequence whose rows include `row` (wave-uniform): the number of i in
// [1, B) with cu[i] <= row, found with 64 probes a step (one load for up to
// 64 sequences, two for 4096) instead of a chain of halvings.
__device__ __forceinline__ int64_t find_sequence(const int32_t *cu, int64_t B, int64_t row) {
    const int lane = threadIdx.x % kWave;
    int64_t lo = 0, n = B - 1;
    while (n > 0) {
        const int64_t step = (n + 63) / 64;
        const int64_t off = (int64_t)(lane + 1) * step;
        const bool below = off <= n && (int64_t)cu[lo + off] <= row;
        const int64_t c = __popcll(__ballot(below));
        lo += c * step;
        n = min(step - 1, n - c * step);
    }
    return lo;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two floats rounded to bf16 (half to even), packed.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const f32x2 f = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
}

template <bool FP32>
__device__ __forceinline__ void load8(const void *x, int64_t at, bool vec, float (&f)[8]) {
    if constexpr (FP32) {
        const float *s = reinterpret_cast<const float *>(x) + at;
        if (vec) {
            const float4 a = *reinterpret_cast<const float4 *>(s);
            const float4 b = *reinterpret_cast<const float4 *>(s + 4);
            f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
            f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = s[j];
        }
    } else {
        const uint16_t *s = reinterpret_cast<const uint16_t *>(x) + at;
        if (vec) {
            const uint4 a = *reinterpret_cast<const uint4 *>(s);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) f[2 * j] = bf16_lo(w[j]), f[2 * j + 1] = bf16_hi(w[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = __uint_as_float((uint32_t)s[j] << 16);
        }
    }
}

// Rounding to the cache's type happens once, here: bf16 half to even, or int8 with
// the scale absmax * fl(1 / 127) of the head's vector (one multiplication, within
// one unit in the last place of the quotient) and codes rne(fl(x / scale)).  A
// vector with a value that is not finite has no int8 form: its scale is NaN.
// `on`: this lane has values of a vector with a place; LPV lanes share a vector.
template <bool INT8, int LPV>
__device__ __forceinline__ void kv_store8(const KvView &c, bool isv, int64_t vec, int d, bool on,
                                          const float (&f)[8]) {
    uint8_t *pool = isv ? c.v : c.k;
    if constexpr (INT8) {
        // the bits of |x| order as the values do, infinity and NaN above them all
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = LPV / 2; o >= 1; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, kWave));
        if (!on) return;
        const float s = m < 0x7F800000u ? __uint_as_float(m) * (1.0f / 127.0f) : NAN;
        uint32_t w[2] = {};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j / 4] |= (uint32_t)(quant_code(f[j], s, -128.0f, 127.0f) & 0xFF) << (j % 4 * 8);
        *reinterpret_cast<uint2 *>(pool + vec * c.D + d) = uint2{w[0], w[1]};
        if (d == 0) (isv ? c.vs : c.ks)[vec] = s;
    } else {
        if (!on) return;
        const u32x4 o = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                         pack_bf16(f[6], f[7])};
        __builtin_nontemporal_store(o, reinterpret_cast<u32x4 *>(pool + (vec * c.D + d) * 2));
    }
}

}  // namespace w4
