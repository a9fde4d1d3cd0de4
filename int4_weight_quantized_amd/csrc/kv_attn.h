// Shared by the attention kernels over the paged key-value cache.
#pragma once

#include <algorithm>

#include "kv_common.h"

namespace w4 {

size_t kv_decode_ws_bytes(int64_t hq, int64_t heads, int64_t D);
hipError_t launch_kv_decode(const KvAttnArgs &a, const char **path, hipStream_t st);
size_t kv_prefill_ws_bytes(int64_t T, int64_t hq, int64_t heads, int64_t D);
hipError_t launch_kv_prefill(const KvAttnArgs &a, const char **path, hipStream_t st);

// Two int8 codes as a bf16 pair: 8 bits are exact in bf16, so the upper halves
// of the two floats are the values.
__device__ __forceinline__ uint32_t code_pair(int lo, int hi) {
    return __builtin_amdgcn_perm(__float_as_uint((float)hi), __float_as_uint((float)lo),
                                 0x07060302u);
}

// Codes 8 half .. 8 half + 7 of 16 bytes as eight bf16.
__device__ __forceinline__ uint4 codes8(const uint4 &w, int half) {
    const uint32_t a = half ? w.z : w.x, b = half ? w.w : w.y;
    return uint4{code_pair((int8_t)a, (int8_t)(a >> 8)),
                 code_pair((int8_t)(a >> 16), (int8_t)(a >> 24)),
                 code_pair((int8_t)b, (int8_t)(b >> 8)),
                 code_pair((int8_t)(b >> 16), (int8_t)(b >> 24))};
}

// Eight floats as N bf16 terms, p = p[0] + p[1] + ..., each the rounding of
// what the terms before it leave: 8 significant bits a term.
template <int N>
__device__ __forceinline__ void split_bf16(const float (&f)[8], uint4 (&out)[N]) {
    float r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = f[j];
#pragma unroll
    for (int t = 0; t < N; ++t) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = pack_bf16(r[2 * j], r[2 * j + 1]);
            r[2 * j] -= bf16_lo(w[j]);
            r[2 * j + 1] -= bf16_hi(w[j]);
        }
        out[t] = uint4{w[0], w[1], w[2], w[3]};
    }
}

// Eight values of q (zeros where !on) as operand terms t, step s.
template <bool FP32, int N, int S>
__device__ __forceinline__ void load_query(const void *q, int64_t at, bool on, uint4 (&out)[N][S],
                                           int s) {
    if constexpr (FP32) {
        float f[8] = {};
        if (on) {
            const float *p = reinterpret_cast<const float *>(q) + at;
            const float4 a = *reinterpret_cast<const float4 *>(p);
            const float4 b = *reinterpret_cast<const float4 *>(p + 4);
            f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
            f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
        }
        uint4 t[N];
        split_bf16<N>(f, t);
#pragma unroll
        for (int i = 0; i < N; ++i) out[i][s] = t[i];
    } else {
        out[0][s] = uint4{};
        if (on)
            out[0][s] = *reinterpret_cast<const uint4 *>(
                reinterpret_cast<const uint16_t *>(q) + at);
    }
}

// Four outputs y / l (zeros where nothing was visible), rounded once.
template <bool FP32>
__device__ __forceinline__ void store_out(void *out, int64_t at, float4 y, float l) {
    const float i = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
    y.x *= i, y.y *= i, y.z *= i, y.w *= i;
    if constexpr (FP32)
        *reinterpret_cast<float4 *>(reinterpret_cast<float *>(out) + at) = y;
    else
        *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(out) + at) =
            uint2{pack_bf16(y.x, y.y), pack_bf16(y.z, y.w)};
}

// Length of sequence b: positions are 32-bit.
constexpr int64_t kMaxLength = (int64_t)1 << 30;
__device__ __forceinline__ int kv_length(const KvAttnArgs &a, int64_t b) {
    return min(max(a.lens[b], 0), (int)min(a.c.W << a.c.shift, kMaxLength));
}

// (m, l, y) += another part (mk, lk, z) of the same row.  A part without a
// maximum is empty (zeros) or has seen nothing but NaN: its sums are added as they
// stand, so that the NaN reaches the row.
__device__ __forceinline__ void add_part(float &m, float &l, float4 &y, float mk, float lk,
                                         float4 z) {
    const float mn = fmaxf(m, mk);
    const float fa = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - mn);
    const float fb = mk == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(mk - mn);
    m = mn;
    l = l * fa + lk * fb;
    y.x = y.x * fa + z.x * fb;
    y.y = y.y * fa + z.y * fb;
    y.z = y.z * fa + z.z * fb;
    y.w = y.w * fa + z.w * fb;
}

// First vector (page, head, slot) of the 16 tokens from `token` on.
__device__ __forceinline__ int64_t kv_vector(const KvView &c, int page, int head, int64_t token) {
    return (((int64_t)page * c.heads + head) << c.shift) + (token & ((1 << c.shift) - 1));
}

}  // namespace w4
