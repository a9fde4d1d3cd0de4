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

// A head's vector into its place; rounding to the cache's type happens once, here:
// bf16 half to even, or int8 with the scale absmax * fl(1 / 127) of the vector (one
// multiplication, within one unit in the last place of the quotient) and codes
// rne(fl(x / scale)), whose quotients are correctly rounded without a division.  A
// vector with a value that is not finite has no int8 form: its scale is NaN.
// LPV lanes share a vector, V values a lane (d: the lane's first); `on`: this lane has
// values of a vector with a place.
template <bool INT8, int V, int LPV>
__device__ __forceinline__ void kv_store(const KvView &c, bool isv, int64_t vec, int d, bool on,
                                         const float (&f)[V]) {
    uint8_t *pool = isv ? c.v : c.k;
    if constexpr (INT8) {
        // the bits of |x| order as the values do, infinity and NaN above them all
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) m = max(m, __float_as_uint(f[j]) & 0x7FFFFFFFu);
        m = max(m, (uint32_t)dpp<kQuadSwap1>((int)m));
        m = max(m, (uint32_t)dpp<kQuadSwap2>((int)m));
        m = max(m, (uint32_t)dpp<kRowHalfMirror>((int)m));
        if constexpr (LPV > 8) m = max(m, (uint32_t)dpp<kRowMirror>((int)m));
#pragma unroll
        for (int o = 16; o < LPV; o *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, o, kWave));
        if (!on) return;
        const float s = m < 0x7F800000u ? __uint_as_float(m) * (1.0f / 127.0f) : NAN;
        uint32_t w[V / 4] = {};
        auto codes = [&](auto code) {
#pragma unroll
            for (int i = 0; i < V / 4; ++i)
                w[i] = pack4_i8(code(f[4 * i]), code(f[4 * i + 1]), code(f[4 * i + 2]), code(f[4 * i + 3]));
        };
        if (s >= kFastQuotientMinScale) {
            const float rs = 1.0f / s;
            codes([&](float x) { return (int)code_in_low_byte(quotient_rn(x, s, rs)); });
        } else {  // zero, tiny or NaN
            codes([&](float x) { return quant_code(x, s, -128.0f, 127.0f); });
        }
        if constexpr (V == 8) *reinterpret_cast<uint2 *>(pool + vec * c.D + d) = uint2{w[0], w[1]};
        else *reinterpret_cast<uint32_t *>(pool + vec * c.D + d) = w[0];
        if (d == 0) (isv ? c.vs : c.ks)[vec] = s;
    } else {
        if (!on) return;
        typedef uint32_t words __attribute__((ext_vector_type(V / 2)));
        words w;
#pragma unroll
        for (int j = 0; j < V / 2; ++j) w[j] = pack_bf16(f[2 * j], f[2 * j + 1]);
        __builtin_nontemporal_store(w, reinterpret_cast<words *>(pool + (vec * c.D + d) * 2));
    }
}

}  // namespace w4
