// Root-mean-square norm of rows with the residual's addition, in fp32, bf16 or
// int8 with a scale per row:
//   h = fl(x + res), r = fl(1 / sqrt(mean(h^2) + eps)), y = fl(fl(h r) fl(offset + w)),
//   sx = fl(max |y| / 127), code = clamp(rne(fl(y / sx)), -128, 127).
// A square of fp32 is exact in fp64 and the sum's rounding there lies 2^-29
// below fp32's, so r, and with it every code next to a rounding border, is the
// same whichever way a row is split over lanes.  Bound by memory: a row is read
// once, kept in registers between the sum and the output, and written once.
#include "kv_common.h"
#include "layer.h"

namespace w4 {

// ------------------------------------------------------------------ helpers
__device__ __forceinline__ double dpp_double(double v, int which) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    int lo = (int)(uint32_t)b, hi = (int)(uint32_t)(b >> 32);
    switch (which) {
        case 0: lo = dpp<kQuadSwap1>(lo), hi = dpp<kQuadSwap1>(hi); break;
        case 1: lo = dpp<kQuadSwap2>(lo), hi = dpp<kQuadSwap2>(hi); break;
        case 2: lo = dpp<kRowHalfMirror>(lo), hi = dpp<kRowHalfMirror>(hi); break;
        default: lo = dpp<kRowMirror>(lo), hi = dpp<kRowMirror>(hi); break;
    }
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)hi << 32 | (uint32_t)lo);
}

__device__ __forceinline__ double lane_double(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Sum over the 64 lanes of a wave (wave-uniform).
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v += dpp_double(v, i);
    return (lane_double(v, 0) + lane_double(v, 16)) + (lane_double(v, 32) + lane_double(v, 48));
}

__device__ __forceinline__ uint32_t wave_max_bits(uint32_t b) {
    b = max(b, (uint32_t)dpp<kQuadSwap1>((int)b));
    b = max(b, (uint32_t)dpp<kQuadSwap2>((int)b));
    b = max(b, (uint32_t)dpp<kRowHalfMirror>((int)b));
    b = max(b, (uint32_t)dpp<kRowMirror>((int)b));
    const uint32_t r0 = __builtin_amdgcn_readlane((int)b, 0);
    const uint32_t r1 = __builtin_amdgcn_readlane((int)b, 16);
    const uint32_t r2 = __builtin_amdgcn_readlane((int)b, 32);
    const uint32_t r3 = __builtin_amdgcn_readlane((int)b, 48);
    return max(max(r0, r1), max(r2, r3));
}

template <int kWaves>
__device__ __forceinline__ float row_rsqrt(double ss, double *red, int64_t K, float eps) {
    ss = wave_sum(ss);
    if constexpr (kWaves > 1) {
        if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = ss;
        lds_barrier();
        ss = red[0];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) ss += red[i];
    }
    return (float)(1.0 / sqrt(ss / (double)K + (double)eps));
}

// The largest |y| of the row as bits, which order as the values do, infinity and
// NaN above them all; the scale of a row with one of those is NaN.
template <int kWaves>
__device__ __forceinline__ float row_scale_of(uint32_t m, uint32_t *red) {
    m = wave_max_bits(m);
    if constexpr (kWaves > 1) {
        if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = m;
        lds_barrier();
        m = red[0];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) m = max(m, red[i]);
    }
    if (m >= 0x7F800000u) return NAN;
    return m == 0 ? 0.0f : div127(__uint_as_float(m));
}

__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }

// Any K, stride and alignment: the row is read twice (the second time from the
// caches) a value at a time.  A value's sum is written by the thread that has
// read it, in the second pass, so that the sum may be the residual or x.
template <bool FP32, int OUT>
__global__ __launch_bounds__(256) void k_rms_norm_any(NormArgs a) {
    __shared__ double red[4];
    __shared__ uint32_t redm[4];
    const int64_t m = blockIdx.x, K = a.K;
    auto value = [&](const void *p, int64_t at) {
        if constexpr (FP32) return reinterpret_cast<const float *>(p)[at];
        return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(p)[at] << 16);
    };
    auto h = [&](int64_t k) {
        const float x = value(a.x, m * a.ldx + k);
        return a.res ? x + value(a.res, m * K + k) : x;
    };
    double ss = 0.0;
    for (int64_t k = threadIdx.x; k < K; k += 256) {
        const double d = h(k);
        ss = __builtin_fma(d, d, ss);
    }
    const float r = row_rsqrt<4>(ss, red, K, a.eps);
    auto y = [&](int64_t k, float v) { return (v * r) * (a.offset + (a.weight ? a.weight[k] : 1.0f)); };
    float s = 0.0f;
    if constexpr (OUT == kNormInt8) {
        uint32_t top = 0;
        for (int64_t k = threadIdx.x; k < K; k += 256) top = max(top, abs_bits(y(k, h(k))));
        s = row_scale_of<4>(top, redm);
        if (threadIdx.x == 0) a.sx[m] = s;
    }
    const RowScale q = row_scale(s);
    for (int64_t k = threadIdx.x; k < K; k += 256) {
        const float v = h(k), f = y(k, v);
        if (a.sum) {
            if constexpr (FP32) reinterpret_cast<float *>(a.sum)[m * K + k] = v;
            else reinterpret_cast<uint16_t *>(a.sum)[m * K + k] = (uint16_t)pack_bf16(v, 0.0f);
        }
        if constexpr (OUT == kNormInt8)
            reinterpret_cast<int8_t *>(a.out)[m * K + k] = (int8_t)quant_code_row(f, q);
        else if constexpr (OUT == RMS_FP32) reinterpret_cast<float *>(a.out)[m * K + k] = f;
        else reinterpret_cast<uint16_t *>(a.out)[m * K + k] = (uint16_t)pack_bf16(f, 0.0f);
    }
}

template <bool FP32>
static void go(const NormArgs &a, hipStream_t st) {
    const dim3 g((unsigned)a.M), b(256);
    if (a.out_type == kNormInt8) launch_kv(k_rms_norm_any<FP32, kNormInt8>, g, b, 0, st, a);
    else if (a.out_type == RMS_FP32) launch_kv(k_rms_norm_any<FP32, RMS_FP32>, g, b, 0, st, a);
    else launch_kv(k_rms_norm_any<FP32, RMS_BF16>, g, b, 0, st, a);
}

hipError_t launch_rms_norm(const NormArgs &a, const char **path, hipStream_t st) {
    *path = "rms_norm";
    if (a.fp32) go<true>(a, st);
    else go<false>(a, st);
    return hipGetLastError();
}

}  // namespace w4
