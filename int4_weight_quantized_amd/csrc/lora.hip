// Low-rank adapters beside a shared product:
//   Y[m] += scale_a ((X[m] A_a^T) B_a^T), a = ids[m].
// Two launches: S = X A^T into the workspace, then Y += scale S B^T.
#include "kv_common.h"
#include "layer.h"

namespace w4 {

// The adapter of a row, or -1.
__device__ __forceinline__ int lora_id(const LoraArgs &a, int64_t m) {
    const int id = a.ids[m];
    return (uint32_t)id < (uint32_t)a.adapters ? id : -1;
}

__device__ __forceinline__ int lora_rank(const LoraArgs &a, int id) {
    return a.ranks ? min(max(a.ranks[id], 0), a.rank) : a.rank;
}

__device__ __forceinline__ float bf16_value(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

__device__ __forceinline__ float wave_add(float v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, kWave);
    return v;
}

// Any sizes and alignment.  One wave a row of X and row j = blockIdx.y of A.
template <bool FP32>
__global__ __launch_bounds__(256) void k_lora_down_any(LoraArgs a) {
    const int64_t m = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave;
    const int j = blockIdx.y;
    if (m >= a.M) return;
    const int id = lora_id(a, m);
    if (id < 0 || j >= lora_rank(a, id)) return;
    const uint16_t *row = a.A + ((int64_t)id * a.rank + j) * a.K;
    float acc = 0.0f;
    for (int64_t k = threadIdx.x % kWave; k < a.K; k += kWave) {
        float x;
        if constexpr (FP32) x = reinterpret_cast<const float *>(a.X)[m * a.ldx + k];
        else x = bf16_value(reinterpret_cast<const uint16_t *>(a.X)[m * a.ldx + k]);
        acc = __builtin_fmaf(x, bf16_value(row[k]), acc);
    }
    acc = wave_add(acc);
    if (threadIdx.x % kWave == 0) a.ws[m * a.rank + j] = acc;
}

// One thread an output; rows beyond the grid's in strides of it.
__global__ __launch_bounds__(256) void k_lora_up_any(LoraArgs a) {
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (n >= a.N) return;
    for (int64_t m = blockIdx.y; m < a.M; m += gridDim.y) {
        const int id = lora_id(a, m);
        if (id < 0) continue;
        const int rank = lora_rank(a, id);
        const uint16_t *col = a.B + ((int64_t)id * a.N + n) * a.rank;
        float acc = 0.0f;
        for (int j = 0; j < rank; ++j)
            acc = __builtin_fmaf(a.ws[m * a.rank + j], bf16_value(col[j]), acc);
        float *y = a.Y + m * a.ldy + n;
        *y += (a.scales ? a.scales[id] : 1.0f) * acc;
    }
}

size_t lora_ws_bytes(int64_t M, int64_t, int64_t, int64_t rank) { return (size_t)M * rank * 4; }

hipError_t launch_lora(const LoraArgs &a, const char **path, hipStream_t st) {
    *path = "lora_any";
    const dim3 down((unsigned)((a.M + 3) / 4), (unsigned)a.rank);
    const dim3 up((unsigned)((a.N + 255) / 256), (unsigned)(a.M < 65535 ? a.M : 65535));
    if (a.fp32) launch_kv(k_lora_down_any<true>, down, dim3(256), 0, st, a);
    else launch_kv(k_lora_down_any<false>, down, dim3(256), 0, st, a);
    launch_kv(k_lora_up_any, up, dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace w4
