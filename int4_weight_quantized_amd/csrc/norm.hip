// Root-mean-square norm of rows with the residual's addition, in fp32, bf16 or
// int8 with a scale per row:
//   h = fl(x + res), r = fl(1 / sqrt(mean(h^2) + eps)), y = fl(fl(h r) fl(offset + w)),
//   sx = fl(max |y| / 127), code = clamp(rne(fl(y / sx)), -128, 127).
// A square of fp32 is exact in fp64 and the sum's rounding there lies 2^-29
// below fp32's, so r, and with it every code next to a rounding border, is the
// same whichever way a row is split over lanes, but for a row in about 2^27 whose
// 1 / sqrt(...) lies in the middle between two fp32 values to within that rounding.
// Bound by memory: a row is read once, kept in registers between the sum and the
// output, and written once.
#include <type_traits>

#include "kv_common.h"
#include "layer.h"

namespace w4 {

template <int N> using Int = std::integral_constant<int, N>;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

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
__device__ __forceinline__ float row_rsqrt(double ss, double *red, int64_t K, double eps) {
    ss = wave_sum(ss);
    if constexpr (kWaves > 1) {
        if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = ss;
        lds_barrier();
        ss = red[0];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) ss += red[i];
    }
    return (float)(1.0 / sqrt(ss / (double)K + eps));
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

// V values as they lie in memory, 16 bytes (V = 4 or 8) or a single one, so that a
// load waits for nothing; outside the row's range a load gives zeros and a store
// writes nothing, which leaves no branch between the loads.
template <bool FP32, int V>
struct Piece {
    static constexpr int kSize = V * (FP32 ? 4 : 2);
    std::conditional_t<V == 1, uint32_t, uint4> w;

    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int g) {
        if constexpr (V > 1) w = bload16_nt(r, g * kSize);
        else if constexpr (FP32) w = __builtin_amdgcn_raw_buffer_load_b32(r, g * kSize, 0, 0);
        else w = __builtin_amdgcn_raw_buffer_load_b16(r, g * kSize, 0, 0);
    }
    __device__ __forceinline__ void values(float (&f)[V]) const {
        if constexpr (V == 1) {
            f[0] = __uint_as_float(FP32 ? w : w << 16);
        } else {
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (FP32) f[j] = __uint_as_float(u[j]);
                else f[2 * j] = bf16_lo(u[j]), f[2 * j + 1] = bf16_hi(u[j]);
            }
        }
    }
};

// V values as fp32 or bf16; AUX: cache policy.
template <bool FP32, int AUX, int V>
__device__ __forceinline__ void store_piece(__amdgpu_buffer_rsrc_t r, int g, const float (&f)[V]) {
    const int at = g * V * (FP32 ? 4 : 2);
    if constexpr (V == 1) {
        if constexpr (FP32) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(f[0]), r, at, 0, 0);
        else __builtin_amdgcn_raw_buffer_store_b16((uint16_t)pack_bf16(f[0], 0.0f), r, at, 0, 0);
    } else if constexpr (FP32) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const v4f v{f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]};
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, at + 16 * i, 0, AUX);
        }
    } else if constexpr (V == 8) {
        const u32x4 w{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                      pack_bf16(f[6], f[7])};
        __builtin_amdgcn_raw_buffer_store_b128(w, r, at, 0, AUX);
    } else {
        const u32x2 w{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])};
        __builtin_amdgcn_raw_buffer_store_b64(w, r, at, 0, AUX);
    }
}

// Rows longer than registers hold: read again from the caches for the scale and
// the output, a value at a time, eight loads of each array ahead.  A value's sum is
// written by the thread that has read it, in the last pass, so that the sum may be
// the residual or x.  (200 rows of 70000 to int8 with residual, us: fp32 96, bf16 62;
// one load at a time 131, 154.)
template <bool FP32, int OUT, bool RES>
__global__ __launch_bounds__(1024) void k_rms_norm_long(NormArgs a) {
    constexpr int kX = FP32 ? 4 : 2, U = 8;
    __shared__ double red[16];
    __shared__ uint32_t redm[16];
    const int64_t m = blockIdx.x, K = a.K;
    const auto rx = make_rsrc(reinterpret_cast<const uint8_t *>(a.x) + m * a.ldx * kX, K * kX);
    const auto rr = make_rsrc(reinterpret_cast<const uint8_t *>(a.res) + m * K * kX, K * kX);
    const auto rw = make_rsrc(a.weight, a.weight ? K * 4 : 0);
    // f(k, h, weight) for this thread's values
    auto each = [&](auto weighted, auto f) {
        for (int k = threadIdx.x; k < (int)K; k += 1024 * U) {
            Piece<FP32, 1> x[U], r[U];
            float w[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                x[u].load(rx, k + 1024 * u);
                if constexpr (RES) r[u].load(rr, k + 1024 * u);
                if constexpr (decltype(weighted)::value) w[u] = bloadf(rw, (k + 1024 * u) * 4);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (k + 1024 * u >= (int)K) break;
                float h[1], add[1];
                x[u].values(h);
                if constexpr (RES) {
                    r[u].values(add);
                    h[0] += add[0];
                }
                f((int64_t)(k + 1024 * u), h[0], decltype(weighted)::value && a.weight ? w[u] : 1.0f);
            }
        }
    };
    double ss = 0.0;
    each(std::false_type{}, [&](int64_t, float v, float) {
        const double d = v;
        ss = __builtin_fma(d, d, ss);
    });
    const float r = row_rsqrt<16>(ss, red, K, a.eps);
    auto y = [&](float v, float w) { return (v * r) * (a.offset + w); };
    float s = 0.0f;
    if constexpr (OUT == kNormInt8) {
        uint32_t top = 0;
        each(std::true_type{}, [&](int64_t, float v, float w) { top = max(top, abs_bits(y(v, w))); });
        s = row_scale_of<16>(top, redm);
        if (threadIdx.x == 0) a.sx[m] = s;
    }
    const RowScale q = row_scale(s);
    each(std::true_type{}, [&](int64_t k, float v, float w) {
        const float f = y(v, w);
        if constexpr (RES) {
            if constexpr (FP32) reinterpret_cast<float *>(a.sum)[m * K + k] = v;
            else reinterpret_cast<uint16_t *>(a.sum)[m * K + k] = (uint16_t)pack_bf16(v, 0.0f);
        }
        if constexpr (OUT == kNormInt8)
            reinterpret_cast<int8_t *>(a.out)[m * K + k] = (int8_t)quant_code_row(f, q);
        else if constexpr (OUT == RMS_FP32) reinterpret_cast<float *>(a.out)[m * K + k] = f;
        else reinterpret_cast<uint16_t *>(a.out)[m * K + k] = (uint16_t)pack_bf16(f, 0.0f);
    });
}

// Pieces of 16 bytes of x, or single values (V = 1) where K, a stride or an address
// does not allow those: thread t owns pieces t, t + T, ... (NG), all loads issued at
// once, neighbouring lanes side by side in every array; a row is read once and stays
// in registers.  x and the residual are read, and the sum written, past the caches,
// whose place the output has for the product that takes it (8192 rows of 8192, fp32
// with residual to bf16, 940 MB: 141 us, 6.7 TB/s; the output past them too 152, all
// through them 160; one row of 1152 to int8 2.1 us, 64 rows of 4096 with residual 3.5;
// single values: 8192 rows of 4097 bf16 65, waiting for each load 142).
// Rows of one wave (T = 64) share a workgroup of four and no barrier.
template <bool FP32, int OUT, bool RES, int V, int T, int NG>
__global__ __launch_bounds__(T > 256 ? T : 256) void k_rms_norm(NormArgs a) {
    constexpr int kWaves = T / kWave, kRows = T > kWave ? 1 : 4;
    constexpr int kX = FP32 ? 4 : 2, kOut = OUT == kNormInt8 ? 1 : OUT == RMS_FP32 ? 4 : 2;
    __shared__ double red[kWaves];
    __shared__ uint32_t redm[kWaves];
    const int in_group = kRows > 1 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x / T) : 0;
    const int64_t m = (int64_t)blockIdx.x * kRows + in_group, K = a.K;
    const int tid = threadIdx.x % T;
    if (kRows > 1 && m >= a.M) return;
    const auto rx = make_rsrc(reinterpret_cast<const uint8_t *>(a.x) + m * a.ldx * kX, K * kX);
    const auto rr = make_rsrc(reinterpret_cast<const uint8_t *>(a.res) + m * K * kX, K * kX);
    const auto rs = make_rsrc(reinterpret_cast<const uint8_t *>(a.sum) + m * K * kX, K * kX);
    const auto ro = make_rsrc(reinterpret_cast<const uint8_t *>(a.out) + m * K * kOut, K * kOut);
    const auto rw = make_rsrc(a.weight, a.weight ? K * 4 : 0);
    Piece<FP32, V> x[NG], r[NG];
    float w[NG][V];
#pragma unroll
    for (int u = 0; u < NG; ++u) {
        x[u].load(rx, tid + T * u);
        if constexpr (RES) r[u].load(rr, tid + T * u);
    }
#pragma unroll
    for (int u = 0; u < NG; ++u) {
        const int at = (tid + T * u) * V * 4;
        if constexpr (V == 1) w[u][0] = bloadf(rw, at);
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const float4 p = bloadf4(rw, at + 16 * i);
            w[u][4 * i] = p.x, w[u][4 * i + 1] = p.y, w[u][4 * i + 2] = p.z, w[u][4 * i + 3] = p.w;
        }
    }
    float h[NG][V];
    double ss = 0.0;
#pragma unroll
    for (int u = 0; u < NG; ++u) {
        x[u].values(h[u]);
        if constexpr (RES) {
            float f[V];
            r[u].values(f);
#pragma unroll
            for (int j = 0; j < V; ++j) h[u][j] += f[j];
            store_piece<FP32, kNonTemporal>(rs, tid + T * u, h[u]);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const double d = h[u][j];
            ss = __builtin_fma(d, d, ss);
        }
    }
    const float s = row_rsqrt<kWaves>(ss, red, K, a.eps);
#pragma unroll
    for (int u = 0; u < NG; ++u)
#pragma unroll
        for (int j = 0; j < V; ++j) h[u][j] = (h[u][j] * s) * (a.offset + (a.weight ? w[u][j] : 1.0f));
    if constexpr (OUT == kNormInt8) {
        // (beyond the row y is zero, or NaN as the row's own values are)
        uint32_t top = 0;
#pragma unroll
        for (int u = 0; u < NG; ++u)
#pragma unroll
            for (int j = 0; j < V; ++j) top = max(top, abs_bits(h[u][j]));
        const float sx = row_scale_of<kWaves>(top, redm);
        if (tid == 0) a.sx[m] = sx;
        auto codes = [&](auto code) {
#pragma unroll
            for (int u = 0; u < NG; ++u) {
                const int at = (tid + T * u) * V;
                const float(&f)[V] = h[u];
                if constexpr (V == 1) {
                    __builtin_amdgcn_raw_buffer_store_b8((uint8_t)code(f[0]), ro, at, 0, 0);
                } else {
                    uint32_t c[V / 4];
#pragma unroll
                    for (int i = 0; i < V / 4; ++i)
                        c[i] = pack4_i8(code(f[4 * i]), code(f[4 * i + 1]), code(f[4 * i + 2]),
                                        code(f[4 * i + 3]));
                    if constexpr (V == 8)
                        __builtin_amdgcn_raw_buffer_store_b64(u32x2{c[0], c[1]}, ro, at, 0, 0);
                    else __builtin_amdgcn_raw_buffer_store_b32(c[0], ro, at, 0, 0);
                }
            }
        };
        if (sx >= kFastQuotientMinScale) {
            const float inv = 1.0f / sx;
            codes([&](float v) { return (int)code_in_low_byte(quotient_rn(v, sx, inv)); });
        } else {  // zero, tiny or NaN
            const RowScale q = row_scale(sx);
            codes([&](float v) { return quant_code_row(v, q); });
        }
    } else {
#pragma unroll
        for (int u = 0; u < NG; ++u) store_piece<OUT == RMS_FP32, 0>(ro, tid + T * u, h[u]);
    }
}

template <bool FP32, int OUT>
static void launch_as(const NormArgs &a, const char **path, hipStream_t st) {
    auto at = [](const void *p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
    constexpr int V = FP32 ? 4 : 8;
    const bool whole = a.K % V == 0 && a.ldx % V == 0 && at(a.x, 16) && at(a.res, 16) &&
                       at(a.sum, 16) && at(a.weight, 16) &&
                       at(a.out, OUT == kNormInt8 ? V : OUT == RMS_FP32 ? 16 : 2 * V);
    auto go = [&](auto v, auto t, auto values) {
        constexpr int P = decltype(v)::value, T = decltype(t)::value;
        constexpr int NG = decltype(values)::value / P;
        const dim3 g((unsigned)(T > kWave ? a.M : (a.M + 3) / 4)), b(T > kWave ? T : 256);
        *path = P > 1 ? "rms_norm" : "rms_norm_odd";
        if (a.res) launch_kv(k_rms_norm<FP32, OUT, true, P, T, NG>, g, b, 0, st, a);
        else launch_kv(k_rms_norm<FP32, OUT, false, P, T, NG>, g, b, 0, st, a);
    };
    auto run = [&](auto t, auto values) { go(Int<V>{}, t, values); };
    // Up to 32 values a thread, and the fewest threads that this allows: they meet at
    // fewer barriers (8192 rows of 8192, us: 256 / 512 / 1024 threads 151 / 156 / 153;
    // 64 rows of 4096: 3.6 / 3.6 / 5.2).
    if (whole && a.K <= 512) return run(Int<64>{}, Int<8>{});
    if (whole && a.K <= 2048) return run(Int<256>{}, Int<8>{});
    if (whole && a.K <= 4096) return run(Int<256>{}, Int<16>{});
    if (whole && a.K <= 8192) return run(Int<256>{}, Int<32>{});
    if (whole && a.K <= 16384) return run(Int<512>{}, Int<32>{});
    if (whole && a.K <= 32768) return run(Int<1024>{}, Int<32>{});
    if (!whole && a.K <= 512) return go(Int<1>{}, Int<64>{}, Int<8>{});
    if (!whole && a.K <= 2048) return go(Int<1>{}, Int<256>{}, Int<8>{});
    if (!whole && a.K <= 8192) return go(Int<1>{}, Int<256>{}, Int<32>{});
    if (!whole && a.K <= 16384) return go(Int<1>{}, Int<512>{}, Int<32>{});
    if (!whole && a.K <= 32768) return go(Int<1>{}, Int<1024>{}, Int<32>{});
    *path = "rms_norm_long";
    if (a.res) launch_kv(k_rms_norm_long<FP32, OUT, true>, dim3((unsigned)a.M), dim3(1024), 0, st, a);
    else launch_kv(k_rms_norm_long<FP32, OUT, false>, dim3((unsigned)a.M), dim3(1024), 0, st, a);
}

hipError_t launch_rms_norm(const NormArgs &a, const char **path, hipStream_t st) {
    auto type = [&](auto fp32) {
        constexpr bool F = decltype(fp32)::value;
        if (a.out_type == kNormInt8) launch_as<F, kNormInt8>(a, path, st);
        else if (a.out_type == RMS_FP32) launch_as<F, RMS_FP32>(a, path, st);
        else launch_as<F, RMS_BF16>(a, path, st);
    };
    if (a.fp32) type(std::true_type{});
    else type(std::false_type{});
    return hipGetLastError();
}

}  // namespace w4
