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

}  // namespace w4
