// Host-side launchers of the operators around a decoder layer's quantized
// projections: norms, rotary positions, adapters (internal to the library).
// Arguments are validated by the C ABI layer before any launcher runs; each
// launcher only enqueues work on `st` and returns hipGetLastError().
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/w4.h"
#include "kv.h"

namespace w4 {

struct NormArgs {
    const void *x, *res;  // [M][K], res NULL: none
    bool fp32;            // type of x, res and sum
    int64_t ldx;
    const float *weight;  // NULL: ones
    float offset;
    double eps;
    int64_t M, K;
    void *sum;            // NULL without res
    void *out;            // bf16, fp32 or int8
    int out_type;         // RMS_BF16, RMS_FP32 or kNormInt8
    float *sx;            // int8 only
};
constexpr int kNormInt8 = 2;

// `path`, here and below: the kernel variant taken.
hipError_t launch_rms_norm(const NormArgs &a, const char **path, hipStream_t st);

// Frequencies of a rotation and where it applies (rope_spec).
struct RopeView {
    const double *turns;
    int rot, half;
    bool pairs;
    double magnitude;
};

struct RopeArgs {
    RopeView rope;
    const void *x;
    bool fp32;
    int64_t ldx, T;
    int heads, D;
    const int32_t *pos;
    void *out;
    int64_t ldo;
};

hipError_t launch_rope(const RopeArgs &a, const char **path, hipStream_t st);

struct AppendRopeArgs {
    RopeView rope;
    KvView c;
    bool int8;      // cache codes
    KvRows rows;
    const void *q, *k, *v;
    bool fp32;      // activations
    int64_t ldq, ldk, ldv;
    int hq;
    void *out;
    int64_t ldo;
};

hipError_t launch_kv_append_rope(const AppendRopeArgs &a, const char **path, hipStream_t st);

struct LoraArgs {
    const void *X;
    bool fp32;
    int64_t ldx, M, K, N;
    const int32_t *ids;
    const uint16_t *A, *B;
    int64_t adapters;
    int rank;
    const float *scales;   // NULL: ones
    const int32_t *ranks;  // NULL: rank
    float *Y;
    int64_t ldy;
    float *ws;
};

size_t lora_ws_bytes(int64_t M, int64_t K, int64_t N, int64_t rank);
hipError_t launch_lora(const LoraArgs &a, const char **path, hipStream_t st);

}  // namespace w4
