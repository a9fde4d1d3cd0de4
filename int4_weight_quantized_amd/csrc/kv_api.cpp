// C ABI of the paged key-value cache: argument checks (pure host code, before
// anything is launched) and the calls of the launchers.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/w4.h"
#include "kv.h"

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxInt = 0x7FFFFFFF;
constexpr int64_t kMaxValues = (int64_t)1 << 46;  // values of K in a cache
// a grid dimension holds fewer than 2^32 threads: rows of a call (256 threads
// each at most) and token-head vectors (32 threads each at most)
constexpr int64_t kMaxRows = (int64_t)1 << 23;
constexpr int64_t kMaxTokens = (int64_t)1 << 30;  // of one sequence
constexpr int64_t kMaxQueries = (int64_t)1 << 28;  // (token, query head) pairs of a call
constexpr int64_t kMaxPairs = (int64_t)1 << 22;    // (sequence, query head) pairs
constexpr int64_t kMaxVectors = (int64_t)1 << 26;

// a * b, or kMaxValues + 1 where it is more (a, b >= 1)
int64_t capped(int64_t a, int64_t b) { return a > kMaxValues / b ? kMaxValues + 1 : a * b; }

int log2_page(int64_t page_size) {
    for (int s = 4; s <= 12; ++s)
        if (page_size == (int64_t)1 << s) return s;
    return -1;
}

int check_cache(const kv_cache *c) {
    if (!c || !c->k || !c->v) return W4_ERR_NULL;
    if (c->dtype != KV_BF16 && c->dtype != KV_INT8) return W4_ERR_ARG;
    if (c->dtype == KV_INT8 && (!c->k_scale || !c->v_scale)) return W4_ERR_NULL;
    if (c->dtype == KV_BF16 && (c->k_scale || c->v_scale)) return W4_ERR_ARG;
    if (c->layers < 1 || c->pages < 1 || c->heads < 1 || c->layers > kMaxInt ||
        c->pages > kMaxInt || c->heads > 65535)
        return W4_ERR_SHAPE;
    if (log2_page(c->page_size) < 0) return W4_ERR_SHAPE;
    if (c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16 != 0) return W4_ERR_SHAPE;
    if (capped(capped(c->layers, c->pages), c->heads * c->page_size * c->head_dim) > kMaxValues)
        return W4_ERR_SHAPE;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) ||
        !aligned(c->v_scale, 16))
        return W4_ERR_ALIGN;
    return W4_OK;
}

// A page table of n rows of W entries.
int check_table(const int32_t *table, int64_t n, int64_t W) {
    if (!table) return W4_ERR_NULL;
    if (n < 1 || W < 1 || n > kMaxInt || W > kMaxInt || n > kMaxInt / W) return W4_ERR_SHAPE;
    if (!aligned(table, 4)) return W4_ERR_ALIGN;
    return W4_OK;
}

int check_workspace(const void *ws, size_t bytes, size_t need, size_t align) {
    if (!ws || bytes < need) return W4_ERR_WORKSPACE;
    return aligned(ws, align) ? W4_OK : W4_ERR_ALIGN;
}

w4::KvView layer_view(const kv_cache *c, int64_t layer, const int32_t *table, int64_t W) {
    const int64_t vecs = c->pages * c->heads * c->page_size;
    const int64_t bytes = vecs * c->head_dim * (c->dtype == KV_BF16 ? 2 : 1);
    w4::KvView v{};
    v.k = static_cast<uint8_t *>(c->k) + layer * bytes;
    v.v = static_cast<uint8_t *>(c->v) + layer * bytes;
    v.ks = c->k_scale ? c->k_scale + layer * vecs : nullptr;
    v.vs = c->v_scale ? c->v_scale + layer * vecs : nullptr;
    v.table = table;
    v.W = W;
    v.pages = (int)c->pages;
    v.heads = (int)c->heads;
    v.D = (int)c->head_dim;
    v.shift = log2_page(c->page_size);
    return v;
}

w4::KvPlanes planes(const kv_cache *c) {
    const int64_t vecs = c->heads * c->page_size;
    w4::KvPlanes p{};
    p.k = static_cast<uint8_t *>(c->k);
    p.v = static_cast<uint8_t *>(c->v);
    p.ks = c->k_scale;
    p.vs = c->v_scale;
    p.layers = c->layers;
    p.pages = c->pages;
    p.page_bytes = vecs * c->head_dim * (c->dtype == KV_BF16 ? 2 : 1);
    p.scale_bytes = c->dtype == KV_INT8 ? vecs * 4 : 0;
    return p;
}

hipStream_t hip_stream(void *s) { return reinterpret_cast<hipStream_t>(s); }

// Checks shared by kv_append and kv_gather (strides in elements).
int check_rows(const kv_cache *c, int64_t layer, const void *k, const void *v, int x_dtype,
               int64_t ldk, int64_t ldv, int64_t T, int64_t B, const int32_t *table, int64_t W,
               const int32_t *start, const int32_t *cu, size_t align) {
    int rc = check_cache(c);
    if (rc != W4_OK) return rc;
    if (!k || !v || !start) return W4_ERR_NULL;
    if ((rc = check_table(table, B, W)) != W4_OK) return rc;
    if (x_dtype != KV_X_BF16 && x_dtype != KV_X_FP32) return W4_ERR_ARG;
    if (layer < 0 || layer >= c->layers) return W4_ERR_ARG;
    const int64_t row = c->heads * c->head_dim;
    if (T < 1 || T > kMaxVectors / c->heads || (!cu && T != B)) return W4_ERR_SHAPE;
    if (ldk < row || ldv < row || ldk > kMaxValues / T || ldv > kMaxValues / T)
        return W4_ERR_SHAPE;
    if (!aligned(k, align) || !aligned(v, align) || !aligned(start, 4) || !aligned(cu, 4))
        return W4_ERR_ALIGN;
    return W4_OK;
}

int attention(const kv_cache *c, int64_t layer, const void *q, int x_dtype,
              int64_t ldq, int64_t T, int64_t B, int64_t hq, const int32_t *table, int64_t W,
              const int32_t *lens, const int32_t *cu, float scale, int64_t window, int64_t sinks,
              void *out, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_cache(c);
    if (rc != W4_OK) return rc;
    if (!q || !out || !lens) return W4_ERR_NULL;
    if ((rc = check_table(table, B, W)) != W4_OK) return rc;
    if (x_dtype != KV_X_BF16 && x_dtype != KV_X_FP32) return W4_ERR_ARG;
    if (layer < 0 || layer >= c->layers || window < 0 || sinks < 0 || !std::isfinite(scale))
        return W4_ERR_ARG;
    if (T < 1 || T > kMaxRows || hq < 1 || hq % c->heads != 0 || hq > 65535 ||
        T > kMaxQueries / hq || B > kMaxPairs / hq)
        return W4_ERR_SHAPE;
    if (ldq < hq * c->head_dim || ldq > kMaxValues / T) return W4_ERR_SHAPE;
    const size_t esize = x_dtype == KV_X_FP32 ? 4 : 2;
    if (!aligned(q, 16) || !aligned(out, 16) || (ldq * (int64_t)esize) % 16 != 0 ||
        !aligned(lens, 4) || !aligned(cu, 4))
        return W4_ERR_ALIGN;
    rc = check_workspace(workspace, workspace_bytes,
                         kv_attention_workspace_bytes(T, B, hq, c->heads, c->head_dim), 256);
    if (rc != W4_OK) return rc;
    w4::KvAttnArgs a{};
    a.c = layer_view(c, layer, table, W);
    a.int8 = c->dtype == KV_INT8;
    a.fp32 = x_dtype == KV_X_FP32;
    a.q = q;
    a.ldq = ldq;
    a.out = out;
    a.lens = lens;
    a.cu = cu;
    a.T = T;
    a.B = B;
    a.hq = (int)hq;
    a.scale = scale;
    a.window = (int)std::min(window, kMaxTokens);
    a.sinks = (int)std::min(sinks, kMaxTokens);
    a.ws = workspace;
    const char *path = "none";
    const hipError_t e = w4::launch_kv_attention(a, &path, hip_stream(stream));
    return w4::finish_call(path, e);
}

}  // namespace

extern "C" {

int kv_append(const kv_cache *cache, int64_t layer, const void *k, const void *v, int x_dtype,
              int64_t k_stride, int64_t v_stride, int64_t T, int64_t B, const int32_t *table,
              int64_t W, const int32_t *start, const int32_t *cu, void *stream) {
    const int rc = check_rows(cache, layer, k, v, x_dtype, k_stride, v_stride, T, B, table, W,
                              start, cu, x_dtype == KV_X_FP32 ? 4 : 2);
    if (rc != W4_OK) return rc;
    const w4::KvRows rows{start, cu, T, B};
    return w4::finish_call(
        "kv_append", w4::launch_kv_append(layer_view(cache, layer, table, W),
                                          cache->dtype == KV_INT8, rows, k, v,
                                          x_dtype == KV_X_FP32, k_stride, v_stride,
                                          hip_stream(stream)));
}

int kv_gather(const kv_cache *cache, int64_t layer, void *k, void *v, int x_dtype, int64_t T,
              int64_t B, const int32_t *table, int64_t W, const int32_t *start,
              const int32_t *cu, void *stream) {
    const int64_t row = cache ? cache->heads * cache->head_dim : 0;
    const int rc = check_rows(cache, layer, k, v, x_dtype, row, row, T, B, table, W, start, cu,
                              16);
    if (rc != W4_OK) return rc;
    const w4::KvRows rows{start, cu, T, B};
    return w4::finish_call(
        "kv_gather", w4::launch_kv_gather(layer_view(cache, layer, table, W),
                                          cache->dtype == KV_INT8, rows, k, v,
                                          x_dtype == KV_X_FP32, hip_stream(stream)));
}

size_t kv_attention_workspace_bytes(int64_t rows, int64_t B, int64_t q_heads, int64_t heads,
                                    int64_t head_dim) {
    if (rows < 1 || B < 1 || q_heads < 1 || heads < 1 || head_dim < 16 || head_dim > 256 ||
        head_dim % 16 != 0 || q_heads % heads != 0 || q_heads > 65535 ||
        rows > kMaxRows || rows > kMaxQueries / q_heads || B > kMaxPairs / q_heads)
        return 0;
    return w4::kv_attn_ws_bytes(rows, q_heads, heads, head_dim);
}

int kv_decode_attention(const kv_cache *cache, int64_t layer, const void *q, int x_dtype,
                        int64_t q_stride, int64_t B, int64_t q_heads, const int32_t *table,
                        int64_t W, const int32_t *lens, float scale, int64_t window,
                        int64_t sinks, void *out, void *workspace, size_t workspace_bytes,
                        void *stream) {
    return attention(cache, layer, q, x_dtype, q_stride, B, B, q_heads, table, W,
                     lens, nullptr, scale, window, sinks, out, workspace, workspace_bytes,
                     stream);
}

int kv_prefill_attention(const kv_cache *cache, int64_t layer, const void *q, int x_dtype,
                         int64_t q_stride, int64_t T, int64_t B, int64_t q_heads,
                         const int32_t *table, int64_t W, const int32_t *lens,
                         const int32_t *cu, float scale, int64_t window, int64_t sinks,
                         void *out, void *workspace, size_t workspace_bytes, void *stream) {
    if (!cu) return W4_ERR_NULL;
    return attention(cache, layer, q, x_dtype, q_stride, T, B, q_heads, table, W,
                     lens, cu, scale, window, sinks, out, workspace, workspace_bytes, stream);
}

int kv_copy_pages(const kv_cache *dst, const int32_t *dst_ids, const kv_cache *src,
                  const int32_t *src_ids, int64_t n, void *stream) {
    int rc = check_cache(dst);
    if (rc == W4_OK) rc = check_cache(src);
    if (rc != W4_OK) return rc;
    if (!dst_ids || !src_ids) return W4_ERR_NULL;
    if (dst->layers != src->layers || dst->heads != src->heads ||
        dst->page_size != src->page_size || dst->head_dim != src->head_dim || n < 1 ||
        n > kMaxRows)
        return W4_ERR_SHAPE;
    if (dst->dtype != src->dtype) return W4_ERR_ARG;
    if (!aligned(dst_ids, 4) || !aligned(src_ids, 4)) return W4_ERR_ALIGN;
    return w4::finish_call("kv_copy_pages",
                           w4::launch_kv_copy_pages(planes(dst), dst_ids, planes(src), src_ids, n,
                                                    hip_stream(stream)));
}

int kv_reserve(int32_t *table, int64_t S, int64_t W, const int32_t *lens, int32_t *refs,
               int64_t pages, int64_t page_size, const int32_t *add, int32_t *ok,
               void *workspace, size_t workspace_bytes, void *stream) {
    if (!lens || !refs || !add || !ok) return W4_ERR_NULL;
    int rc = check_table(table, S, W);
    if (rc != W4_OK) return rc;
    if (pages < 1 || pages > kMaxInt || log2_page(page_size) < 0) return W4_ERR_SHAPE;
    if (!aligned(lens, 4) || !aligned(refs, 4) || !aligned(add, 4) || !aligned(ok, 4))
        return W4_ERR_ALIGN;
    rc = check_workspace(workspace, workspace_bytes, 8 * (size_t)S + 256, 16);
    if (rc != W4_OK) return rc;
    return w4::finish_call("kv_reserve",
                           w4::launch_kv_reserve(table, S, W, lens, refs, pages,
                                                 log2_page(page_size), add, ok,
                                                 static_cast<int32_t *>(workspace),
                                                 hip_stream(stream)));
}

int kv_fork(const kv_cache *cache, int32_t *table, int64_t S, int64_t W, int32_t *lens,
            int32_t *refs, const int32_t *parents, const int32_t *children, int64_t n,
            int32_t *ok, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_cache(cache);
    if (rc != W4_OK) return rc;
    if (!lens || !refs || !parents || !children || !ok) return W4_ERR_NULL;
    if ((rc = check_table(table, S, W)) != W4_OK) return rc;
    if (n < 1 || n > kMaxRows) return W4_ERR_SHAPE;
    if (!aligned(lens, 4) || !aligned(refs, 4) || !aligned(parents, 4) ||
        !aligned(children, 4) || !aligned(ok, 4))
        return W4_ERR_ALIGN;
    rc = check_workspace(workspace, workspace_bytes, 16 * (size_t)n + 256, 16);
    if (rc != W4_OK) return rc;
    return w4::finish_call("kv_fork",
                           w4::launch_kv_fork(planes(cache), log2_page(cache->page_size), table,
                                              S, W, lens, refs, parents, children, n, ok,
                                              static_cast<int32_t *>(workspace),
                                              hip_stream(stream)));
}

int kv_free(int32_t *table, int64_t S, int64_t W, int32_t *lens, int32_t *refs, int64_t pages,
            const int32_t *slots, int64_t n, void *stream) {
    if (!lens || !refs || !slots) return W4_ERR_NULL;
    const int rc = check_table(table, S, W);
    if (rc != W4_OK) return rc;
    if (n < 1 || n > kMaxRows || pages < 1 || pages > kMaxInt) return W4_ERR_SHAPE;
    if (!aligned(lens, 4) || !aligned(refs, 4) || !aligned(slots, 4)) return W4_ERR_ALIGN;
    return w4::finish_call("kv_free", w4::launch_kv_free(table, S, W, lens, refs, pages, slots, n,
                                                         hip_stream(stream)));
}

int kv_compact(const kv_cache *cache, const int32_t *table, int64_t S, int64_t W,
               const int32_t *refs, int32_t *table_out, int32_t *refs_out, int32_t *live,
               void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_cache(cache);
    if (rc != W4_OK) return rc;
    if (!refs || !table_out || !refs_out || !live) return W4_ERR_NULL;
    if ((rc = check_table(table, S, W)) != W4_OK) return rc;
    if (!aligned(refs, 4) || !aligned(table_out, 4) || !aligned(refs_out, 4) || !aligned(live, 4))
        return W4_ERR_ALIGN;
    rc = check_workspace(workspace, workspace_bytes, 8 * (size_t)cache->pages + 256, 16);
    if (rc != W4_OK) return rc;
    return w4::finish_call("kv_compact",
                           w4::launch_kv_compact(planes(cache), table, S, W, refs, table_out,
                                                 refs_out, live, static_cast<int32_t *>(workspace),
                                                 hip_stream(stream)));
}

}  // extern "C"
