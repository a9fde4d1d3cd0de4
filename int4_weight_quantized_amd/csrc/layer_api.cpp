// C ABI of the operators around the quantized projections: argument checks
// (pure host code, before anything is launched), the frequencies of rotary
// positions, and the calls of the launchers.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/w4.h"
#include "layer.h"

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxRows = (int64_t)1 << 23;     // a grid has fewer than 2^32 threads, 256 a row
constexpr int64_t kMaxNorm = (int64_t)1 << 36;     // values of a norm: 512 or 1024 threads a long row
constexpr int64_t kMaxVectors = (int64_t)1 << 26;  // (token, head) pairs of a call
constexpr int64_t kMaxValues = (int64_t)1 << 46;   // of one array, strides included
constexpr int64_t kMaxAdapters = (int64_t)1 << 20;
constexpr int64_t kMaxRank = 256;
constexpr int64_t kMaxInt = 0x7FFFFFFF;

bool x_type(int t) { return t == KV_X_BF16 || t == KV_X_FP32; }
size_t x_size(int t) { return t == KV_X_FP32 ? 4 : 2; }
hipStream_t hip_stream(void *s) { return reinterpret_cast<hipStream_t>(s); }

// T rows of `row` values, `stride` elements apart.
bool rows_ok(int64_t T, int64_t row, int64_t stride) {
    return stride >= row && stride <= kMaxValues / T;
}

int norm(const void *x, int x_dtype, int64_t ldx, const void *res, const float *weight,
         float offset, double eps, int64_t M, int64_t K, void *sum, void *out, int out_type,
         float *sx, void *stream) {
    if (!x || !out || (out_type == w4::kNormInt8 && !sx) || (res != nullptr) != (sum != nullptr))
        return W4_ERR_NULL;
    if (!x_type(x_dtype) || !std::isfinite(offset) || !std::isfinite(eps) || eps < 0.0)
        return W4_ERR_ARG;
    if (M < 1 || K < 1 || M > kMaxRows || K > W4_MAX_K || M > kMaxNorm / K || !rows_ok(M, K, ldx))
        return W4_ERR_SHAPE;
    if (sum == x && ldx != K) return W4_ERR_ARG;  // the sum's rows lie side by side
    const size_t e = x_size(x_dtype);
    const size_t o = out_type == w4::kNormInt8 ? 1 : out_type == RMS_FP32 ? 4 : 2;
    if (!aligned(x, e) || !aligned(res, e) || !aligned(sum, e) || !aligned(weight, 4) ||
        !aligned(out, o) || !aligned(sx, 4))
        return W4_ERR_ALIGN;
    const w4::NormArgs a{x,   res, x_dtype == KV_X_FP32, ldx, weight, offset, eps, M, K, sum,
                         out, out_type, sx};
    const char *path = "none";
    const hipError_t err = w4::launch_rms_norm(a, &path, hip_stream(stream));
    return w4::finish_call(path, err);
}

int check_rope(const rope_spec *r, int64_t head_dim) {
    if (!r || !r->turns) return W4_ERR_NULL;
    if ((r->layout != ROPE_HALF && r->layout != ROPE_PAIRS) || !std::isfinite(r->magnitude))
        return W4_ERR_ARG;
    if (r->rot_dim < 2 || r->rot_dim > 512 || r->rot_dim % 2 != 0 || r->rot_dim > head_dim)
        return W4_ERR_SHAPE;
    return aligned(r->turns, 8) ? W4_OK : W4_ERR_ALIGN;
}

w4::RopeView rope_view(const rope_spec *r) {
    return w4::RopeView{r->turns, (int)r->rot_dim, (int)(r->rot_dim / 2), r->layout == ROPE_PAIRS,
                        r->magnitude};
}

bool lora_sizes(int64_t M, int64_t K, int64_t N, int64_t rank) {
    return M >= 1 && K >= 1 && N >= 1 && rank >= 1 && M <= kMaxRows && K <= W4_MAX_K &&
           N <= kMaxInt && rank <= kMaxRank;
}

}  // namespace

extern "C" {

int rms_norm(const void *x, int x_dtype, int64_t x_stride, const void *residual,
             const float *weight, float offset, double eps, int64_t M, int64_t K, void *sum,
             void *out, int out_dtype, void *stream) {
    if (out_dtype != RMS_BF16 && out_dtype != RMS_FP32) return W4_ERR_ARG;
    return norm(x, x_dtype, x_stride, residual, weight, offset, eps, M, K, sum, out, out_dtype,
                nullptr, stream);
}

int a8_rms_norm(const void *x, int x_dtype, int64_t x_stride, const void *residual,
                const float *weight, float offset, double eps, int64_t M, int64_t K, void *sum,
                int8_t *Xq, float *sx, void *stream) {
    return norm(x, x_dtype, x_stride, residual, weight, offset, eps, M, K, sum, Xq,
                w4::kNormInt8, sx, stream);
}

int rope_frequencies(int64_t rot_dim, double base, int scaling, double factor, int64_t context,
                     double fast, double slow, double *turns, double *magnitude) {
    if (!turns || !magnitude) return W4_ERR_NULL;
    if (rot_dim < 2 || rot_dim > 512 || rot_dim % 2 != 0) return W4_ERR_SHAPE;
    if (!(base > 1.0) || !std::isfinite(base) || scaling < ROPE_PLAIN || scaling > ROPE_BANDS)
        return W4_ERR_ARG;
    if (scaling != ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return W4_ERR_ARG;
    if ((scaling == ROPE_YARN || scaling == ROPE_BANDS) &&
        (context < 1 || !(slow > 0.0) || !(fast > slow) || !std::isfinite(fast)))
        return W4_ERR_ARG;
    constexpr double kTurn = 2.0 * 3.14159265358979323846;
    const double rot = (double)rot_dim;
    // (a single pair turns once in 2 pi tokens whatever the base is)
    if (scaling == ROPE_NTK && rot_dim > 2) base = base * std::pow(factor, rot / (rot - 2.0));
    double low = 0.0, high = 0.0;
    *magnitude = 1.0;
    if (scaling == ROPE_YARN) {
        // the index, not rounded, of the pair that makes `t` turns within the context
        auto index = [&](double t) {
            return rot * std::log((double)context / (kTurn * t)) / (2.0 * std::log(base));
        };
        low = std::max(std::floor(index(fast)), 0.0);
        high = std::min(std::ceil(index(slow)), rot - 1.0);
        *magnitude = 0.1 * std::log(factor) + 1.0;
    }
    for (int64_t i = 0; i < rot_dim / 2; ++i) {
        const double f = std::pow(base, -2.0 * (double)i / rot) / kTurn;
        double keep = 1.0;  // share of the pair's own frequency
        if (scaling == ROPE_YARN) {
            const double ramp =
                std::min(std::max(((double)i - low) / std::max(high - low, 0.001), 0.0), 1.0);
            turns[i] = f / factor * ramp + f * (1.0 - ramp);
            continue;
        }
        if (scaling == ROPE_BANDS)
            keep = std::min(std::max(((double)context * f - slow) / (fast - slow), 0.0), 1.0);
        turns[i] = scaling == ROPE_LINEAR ? f / factor : f * keep + f / factor * (1.0 - keep);
        if (scaling == ROPE_PLAIN || scaling == ROPE_NTK) turns[i] = f;
    }
    return W4_OK;
}

int rope_rotate(const rope_spec *rope, const void *x, int x_dtype, int64_t x_stride, int64_t T,
                int64_t heads, int64_t head_dim, const int32_t *pos, void *out,
                int64_t out_stride, void *stream) {
    int rc = check_rope(rope, head_dim);
    if (rc != W4_OK) return rc;
    if (!x || !pos || !out) return W4_ERR_NULL;
    if (!x_type(x_dtype)) return W4_ERR_ARG;
    if (head_dim > 512 || head_dim % 8 != 0 || T < 1 || T > kMaxRows || heads < 1 ||
        heads > 65535 || heads > kMaxVectors / T || !rows_ok(T, heads * head_dim, x_stride) ||
        !rows_ok(T, heads * head_dim, out_stride))
        return W4_ERR_SHAPE;
    if (x == out && x_stride != out_stride) return W4_ERR_ARG;
    if (!aligned(x, x_size(x_dtype)) || !aligned(out, x_size(x_dtype)) || !aligned(pos, 4))
        return W4_ERR_ALIGN;
    const w4::RopeArgs a{rope_view(rope), x, x_dtype == KV_X_FP32, x_stride, T, (int)heads,
                         (int)head_dim, pos, out, out_stride};
    const char *path = "none";
    const hipError_t e = w4::launch_rope(a, &path, hip_stream(stream));
    return w4::finish_call(path, e);
}

int kv_append_rope(const kv_cache *cache, int64_t layer, const rope_spec *rope, const void *q,
                   const void *k, const void *v, int x_dtype, int64_t q_stride, int64_t k_stride,
                   int64_t v_stride, int64_t q_heads, int64_t T, int64_t B, const int32_t *table,
                   int64_t W, const int32_t *start, const int32_t *cu, void *q_out,
                   int64_t out_stride, void *stream) {
    int rc = w4::check_kv_rows(cache, layer, k, v, x_dtype, k_stride, v_stride, T, B, table, W,
                               start, cu, x_size(x_dtype));
    if (rc == W4_OK) rc = check_rope(rope, cache->head_dim);
    if (rc != W4_OK) return rc;
    if (!q || !q_out) return W4_ERR_NULL;
    if (q_heads < 1 || q_heads > 65535 || T > kMaxRows ||
        q_heads + 2 * cache->heads > kMaxVectors / T ||
        !rows_ok(T, q_heads * cache->head_dim, q_stride) ||
        !rows_ok(T, q_heads * cache->head_dim, out_stride))
        return W4_ERR_SHAPE;
    if (q == q_out && q_stride != out_stride) return W4_ERR_ARG;
    if (!aligned(q, x_size(x_dtype)) || !aligned(q_out, x_size(x_dtype))) return W4_ERR_ALIGN;
    const w4::AppendRopeArgs a{rope_view(rope),
                               w4::kv_layer_view(cache, layer, table, W),
                               cache->dtype == KV_INT8,
                               w4::KvRows{start, cu, T, B},
                               q, k, v,
                               x_dtype == KV_X_FP32,
                               q_stride, k_stride, v_stride,
                               (int)q_heads,
                               q_out, out_stride};
    const char *path = "none";
    const hipError_t e = w4::launch_kv_append_rope(a, &path, hip_stream(stream));
    return w4::finish_call(path, e);
}

size_t lora_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t rank) {
    return lora_sizes(M, K, N, rank) ? w4::lora_ws_bytes(M, K, N, rank) : 0;
}

int lora_add(const void *X, int x_dtype, int64_t x_stride, int64_t M, int64_t K, int64_t N,
             const int32_t *ids, const uint16_t *A, const uint16_t *B, int64_t adapters,
             int64_t rank, const float *scales, const int32_t *ranks, float *Y, int64_t y_stride,
             void *workspace, size_t workspace_bytes, void *stream) {
    if (!X || !ids || !A || !B || !Y) return W4_ERR_NULL;
    if (!x_type(x_dtype)) return W4_ERR_ARG;
    if (!lora_sizes(M, K, N, rank) || adapters < 1 || adapters > kMaxAdapters ||
        adapters * rank > kMaxValues / std::max(K, N) || !rows_ok(M, K, x_stride) ||
        !rows_ok(M, N, y_stride))
        return W4_ERR_SHAPE;
    if (!aligned(X, x_size(x_dtype)) || !aligned(ids, 4) || !aligned(A, 2) || !aligned(B, 2) ||
        !aligned(scales, 4) || !aligned(ranks, 4) || !aligned(Y, 4))
        return W4_ERR_ALIGN;
    if (!workspace || workspace_bytes < w4::lora_ws_bytes(M, K, N, rank)) return W4_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return W4_ERR_ALIGN;
    const w4::LoraArgs a{X, x_dtype == KV_X_FP32, x_stride, M, K, N, ids, A, B, adapters,
                         (int)rank, scales, ranks, Y, y_stride, static_cast<float *>(workspace)};
    const char *path = "none";
    const hipError_t e = w4::launch_lora(a, &path, hip_stream(stream));
    return w4::finish_call(path, e);
}

}  // extern "C"
