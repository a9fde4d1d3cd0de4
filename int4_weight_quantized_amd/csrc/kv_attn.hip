// Attention over the paged key-value cache.
#include <type_traits>

#include "kv_attn.h"

namespace w4 {

size_t kv_attn_ws_bytes(int64_t, int64_t, int64_t hq, int64_t heads, int64_t D) {
    return kv_decode_ws_bytes(hq, heads, D);
}

// One workgroup per query row and head: scores of 256 tokens at a time (one
// token a thread), a running maximum and sum, and the weighted sum of V with
// one output column a thread.
template <bool INT8, bool FP32>
__global__ __launch_bounds__(256) void k_kv_attn_rows(KvAttnArgs a) {
    __shared__ float q[256], p[256], red[4];
    const int tid = threadIdx.x, D = a.c.D;
    const int64_t row = blockIdx.x;
    const int h = blockIdx.y, kvh = h / (a.hq / a.c.heads);
    const int64_t b = a.cu ? find_sequence(a.cu, a.B, row) : row;
    const int64_t cap = a.c.W << a.c.shift;
    const int64_t len = min((int64_t)max(a.lens[b], 0), cap);
    int64_t pos = len - 1;
    if (a.cu) pos = len - ((int64_t)a.cu[b + 1] - row);
    const int64_t at = row * a.ldq + (int64_t)h * D;
    if (tid < D)
        q[tid] = FP32 ? reinterpret_cast<const float *>(a.q)[at + tid]
                      : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(a.q)[at + tid] << 16);
    __syncthreads();
    const int32_t *table = a.c.table + b * a.c.W;
    const int mask = (1 << a.c.shift) - 1;
    float m = -INFINITY, l = 0.0f, o = 0.0f;
    for (int64_t t0 = 0; t0 <= pos; t0 += 256) {
        if (a.window && t0 + 256 <= pos - a.window + 1 && t0 >= a.sinks) continue;
        const int64_t t = t0 + tid;
        bool see = t <= pos && t < len && (!a.window || t > pos - a.window || t < a.sinks);
        const int page = see ? kv_page(a.c, table, t) : -1;
        see = page >= 0;
        const int64_t vec = (((int64_t)page * a.c.heads + kvh) << a.c.shift) + (t & mask);
        float s = -INFINITY;
        if (see) {
            float x = 0.0f;
            for (int d = 0; d < D; ++d) {
                const float kv = INT8 ? (float)reinterpret_cast<const int8_t *>(a.c.k)[vec * D + d]
                                      : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(a.c.k)[vec * D + d] << 16);
                x = __builtin_fmaf(q[d], kv, x);
            }
            s = x * a.scale * (INT8 ? a.c.ks[vec] : 1.0f);
        }
        float mx = wave_max(s);
        if (tid % kWave == 0) red[tid / kWave] = mx;
        __syncthreads();
        const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
        const float alpha = mn == -INFINITY ? 1.0f : expf(m - mn);
        p[tid] = see ? expf(s - mn) : 0.0f;
        __syncthreads();
        m = mn;
        l *= alpha;
        o *= alpha;
        for (int j = 0; j < 256; ++j) {
            if (p[j] == 0.0f) continue;
            l += p[j];
            const int64_t tj = t0 + j;
            const int pg = kv_page(a.c, table, tj);
            const int64_t vj = (((int64_t)pg * a.c.heads + kvh) << a.c.shift) + (tj & mask);
            if (tid < D) {
                const float vv = INT8 ? (float)reinterpret_cast<const int8_t *>(a.c.v)[vj * D + tid] * a.c.vs[vj]
                                      : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(a.c.v)[vj * D + tid] << 16);
                o = __builtin_fmaf(p[j], vv, o);
            }
        }
        __syncthreads();
    }
    if (tid < D) {
        const float y = l > 0.0f ? o / l : 0.0f;
        const int64_t w = (row * a.hq + h) * D + tid;
        if (FP32)
            reinterpret_cast<float *>(a.out)[w] = y;
        else
            reinterpret_cast<__bf16 *>(a.out)[w] = (__bf16)y;
    }
}

hipError_t launch_kv_attention(const KvAttnArgs &a, hipStream_t st) {
    if (!a.cu) return launch_kv_decode(a, st);
    const dim3 g((unsigned)a.T, (unsigned)a.hq);
    if (a.int8 && a.fp32)
        hipLaunchKernelGGL((k_kv_attn_rows<true, true>), g, dim3(256), 0, st, a);
    else if (a.int8)
        hipLaunchKernelGGL((k_kv_attn_rows<true, false>), g, dim3(256), 0, st, a);
    else if (a.fp32)
        hipLaunchKernelGGL((k_kv_attn_rows<false, true>), g, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((k_kv_attn_rows<false, false>), g, dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace w4
