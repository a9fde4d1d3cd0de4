// Rotary positions: a standalone rotation of heads, and one on the way into the
// paged cache (queries rotated, keys rotated and cached, values cached).
// Pair i of a token at position p turns by t = p turns[i] full turns:
//   (a, b) -> (fl(fl(a c) - fl(b s)), fl(fl(b c) + fl(a s))),
//   c, s = fp32 of magnitude * cos, sin(2 pi t).
// Angles are taken in fp64: p turns[i] loses 2^-53 of itself, so that a token at
// position 10^6 still has its angle to 10^-10 where fp32 would be off by a tenth
// of a turn, and c and s are rounded once.  A token's angles are computed once
// by its workgroup, for all of its heads.
#include "kv_common.h"
#include "layer.h"

namespace w4 {

constexpr int kTokens = 4;     // of a workgroup, at most
constexpr int kHalf = 256;     // pairs of a token, at most

struct RopeLds {
    float2 cs[kTokens * kHalf];
    float4 swap[2][256];
};

// Angles of a workgroup's tokens at positions pos[0 .. n - 1] (LDS).
__device__ __forceinline__ void rope_angles(const RopeView &r, const int64_t *pos, int n,
                                            float2 *cs) {
    for (int i = threadIdx.x; i < n * r.half; i += 256) {
        const int t = i / r.half;
        const double turns = (double)pos[t] * r.turns[i - t * r.half];
        double s, c;
        sincospi(2.0 * (turns - rint(turns)), &s, &c);
        cs[i] = float2{(float)(r.magnitude * c), (float)(r.magnitude * s)};
    }
}

// Rotate the 8 values d, d + 1, ... of a head that this lane holds; the other
// half of a pair is another lane's of the same wave, which hands it over in LDS.
__device__ __forceinline__ void rotate8(const RopeView &r, const float2 *cs, int d, float4 (*swap)[256],
                                        float (&f)[8]) {
    if (r.pairs) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            if (d + j >= r.rot) continue;
            const float2 u = cs[(d + j) / 2];
            const float a = f[j], b = f[j + 1];
            f[j] = a * u.x - b * u.y;
            f[j + 1] = b * u.x + a * u.y;
        }
        return;
    }
    swap[0][threadIdx.x] = float4{f[0], f[1], f[2], f[3]};
    swap[1][threadIdx.x] = float4{f[4], f[5], f[6], f[7]};
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int first = threadIdx.x - d / 8;  // the lane of the head's value 0
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int e = d + j;
        if (e >= r.rot) continue;
        const bool low = e < r.half;
        const int o = low ? e + r.half : e - r.half;
        const float other =
            reinterpret_cast<const float *>(&swap[(o >> 2) & 1][first + (o >> 3)])[o & 3];
        const float2 u = cs[low ? e : o];
        f[j] = low ? f[j] * u.x - other * u.y : f[j] * u.x + other * u.y;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

template <bool FP32>
__device__ __forceinline__ void store8(void *x, int64_t at, bool vec, const float (&f)[8]) {
    if constexpr (FP32) {
        float *o = reinterpret_cast<float *>(x) + at;
        if (vec) {
            reinterpret_cast<float4 *>(o)[0] = float4{f[0], f[1], f[2], f[3]};
            reinterpret_cast<float4 *>(o)[1] = float4{f[4], f[5], f[6], f[7]};
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = f[j];
        }
    } else {
        uint16_t *o = reinterpret_cast<uint16_t *>(x) + at;
        const uint4 w = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                         pack_bf16(f[6], f[7])};
        if (vec) {
            *reinterpret_cast<uint4 *>(o) = w;
        } else {
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = (uint16_t)(u[j / 2] >> (j % 2 * 16));
        }
    }
}

// LPV lanes a head, 8 values a lane.
template <bool FP32, int LPV>
__global__ __launch_bounds__(256) void k_rope(RopeArgs a, bool vec) {
    __shared__ RopeLds lds;
    __shared__ int64_t pos[kTokens];
    const int64_t t0 = (int64_t)blockIdx.x * kTokens;
    const int n = (int)min((int64_t)kTokens, a.T - t0);
    if (threadIdx.x < n) pos[threadIdx.x] = a.pos[t0 + threadIdx.x];
    __syncthreads();
    rope_angles(a.rope, pos, n, lds.cs);
    __syncthreads();
    const int d = threadIdx.x % LPV * 8;
    for (int i = 0; i < n * a.heads; i += 256 / LPV) {
        const int v = i + threadIdx.x / LPV;
        const int t = v / a.heads, h = v - t * a.heads;
        const bool on = t < n && d < a.D;
        float f[8] = {};
        if (on) load8<FP32>(a.x, (t0 + t) * a.ldx + (int64_t)h * a.D + d, vec, f);
        rotate8(a.rope, lds.cs + min(t, n - 1) * a.rope.half, d, lds.swap, f);
        if (on) store8<FP32>(a.out, (t0 + t) * a.ldo + (int64_t)h * a.D + d, vec, f);
    }
}

// A token of the call: its position (-1: of no sequence, or skipped) and its
// place in head 0 of its page (-1: it has no page).
struct TokenPlace {
    int64_t pos, at;
};

__device__ __forceinline__ TokenPlace token_place(const KvView &c, const KvRows &r, int64_t row) {
    int64_t b = row, pos = 0;
    if (r.cu) {
        b = find_sequence(r.cu, r.B, row);
        if (row < r.cu[b] || row >= r.cu[b + 1]) return {-1, -1};
        pos = row - r.cu[b];
    }
    const int start = r.start[b];
    if (start < 0) return {-1, -1};
    pos += start;
    const int page = kv_page(c, c.table + b * c.W, pos);
    return {pos, page < 0 ? -1
                          : (((int64_t)page * c.heads) << c.shift) + (pos & ((1 << c.shift) - 1))};
}

template <bool INT8, bool FP32, int LPV>
__global__ __launch_bounds__(256) void k_kv_append_rope(AppendRopeArgs a, bool vecq, bool veckv) {
    __shared__ RopeLds lds;
    __shared__ int64_t pos[kTokens], at[kTokens];
    const int64_t t0 = (int64_t)blockIdx.x * kTokens;
    const int n = (int)min((int64_t)kTokens, a.rows.T - t0);
    const int wave = threadIdx.x / kWave;
    if (wave < n) {
        const TokenPlace p = token_place(a.c, a.rows, t0 + wave);
        if (threadIdx.x % kWave == 0) pos[wave] = p.pos, at[wave] = p.at;
    }
    __syncthreads();
    rope_angles(a.rope, pos, n, lds.cs);
    __syncthreads();
    const int d = threadIdx.x % LPV * 8, D = a.c.D, heads = a.hq + 2 * a.c.heads;
    for (int i = 0; i < n * heads; i += 256 / LPV) {
        const int v = i + threadIdx.x / LPV;
        const int t = min(v / heads, n - 1), h = v - v / heads * heads;
        const bool isq = h < a.hq, isv = h >= a.hq + a.c.heads;
        const int64_t row = t0 + t;
        const int kh = isv ? h - a.hq - a.c.heads : h - a.hq;
        const bool on = v < n * heads && d < D && pos[t] >= 0 && (isq || at[t] >= 0);
        float f[8] = {};
        if (on) {
            if (isq) load8<FP32>(a.q, row * a.ldq + (int64_t)h * D + d, vecq, f);
            else if (isv) load8<FP32>(a.v, row * a.ldv + (int64_t)kh * D + d, veckv, f);
            else load8<FP32>(a.k, row * a.ldk + (int64_t)kh * D + d, veckv, f);
        }
        float g[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = f[j];
        rotate8(a.rope, lds.cs + t * a.rope.half, d, lds.swap, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = isv ? f[j] : g[j];
        if (isq) {
            if (on) store8<FP32>(a.out, row * a.ldo + (int64_t)h * D + d, vecq, f);
        }
        const int64_t vec = at[t] + ((int64_t)max(kh, 0) << a.c.shift);
        kv_store8<INT8, LPV>(a.c, isv, vec, d, on && !isq, f);
    }
}

static bool aligned16(const void *p, int64_t stride, bool fp32) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride * (fp32 ? 4 : 2) % 16 == 0;
}

template <bool FP32>
static void go_rope(const RopeArgs &a, hipStream_t st) {
    const dim3 g((unsigned)((a.T + kTokens - 1) / kTokens)), b(256);
    const bool vec = aligned16(a.x, a.ldx, FP32) && aligned16(a.out, a.ldo, FP32);
    if (a.D <= 64) launch_kv(k_rope<FP32, 8>, g, b, 0, st, a, vec);
    else if (a.D <= 128) launch_kv(k_rope<FP32, 16>, g, b, 0, st, a, vec);
    else if (a.D <= 256) launch_kv(k_rope<FP32, 32>, g, b, 0, st, a, vec);
    else launch_kv(k_rope<FP32, 64>, g, b, 0, st, a, vec);
}

hipError_t launch_rope(const RopeArgs &a, hipStream_t st) {
    if (a.fp32) go_rope<true>(a, st);
    else go_rope<false>(a, st);
    return hipGetLastError();
}

template <bool INT8, bool FP32>
static void go_append(const AppendRopeArgs &a, hipStream_t st) {
    const dim3 g((unsigned)((a.rows.T + kTokens - 1) / kTokens)), b(256);
    const bool vecq = aligned16(a.q, a.ldq, FP32) && aligned16(a.out, a.ldo, FP32);
    const bool veckv = aligned16(a.k, a.ldk, FP32) && aligned16(a.v, a.ldv, FP32);
    if (a.c.D <= 64) launch_kv(k_kv_append_rope<INT8, FP32, 8>, g, b, 0, st, a, vecq, veckv);
    else if (a.c.D <= 128) launch_kv(k_kv_append_rope<INT8, FP32, 16>, g, b, 0, st, a, vecq, veckv);
    else launch_kv(k_kv_append_rope<INT8, FP32, 32>, g, b, 0, st, a, vecq, veckv);
}

hipError_t launch_kv_append_rope(const AppendRopeArgs &a, hipStream_t st) {
    if (a.int8) a.fp32 ? go_append<true, true>(a, st) : go_append<true, false>(a, st);
    else a.fp32 ? go_append<false, true>(a, st) : go_append<false, false>(a, st);
    return hipGetLastError();
}

}  // namespace w4
