// Host-side launchers of the paged key-value cache's kernels (internal to the
// library).  Arguments are validated by the C ABI layer before any launcher
// runs; each launcher only enqueues work on `st` and returns hipGetLastError().
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/w4.h"
#include "kernels.h"

namespace w4 {

// Record the outcome of a launch as the C ABI's status (api.cpp).
int finish_call(const char *path, hipError_t e);

// Launch a call's main kernel, and remember it as the one that the call ran.
template <typename... KArgs, typename... Args>
inline void launch_kv(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t lds, hipStream_t st,
                      Args... args) {
    note_kernel(reinterpret_cast<const void *>(kernel), st);
    hipLaunchKernelGGL(kernel, grid, block, lds, st, KArgs(args)...);
}

// One layer of a cache and the page table of a call, as the kernels take them.
struct KvView {
    uint8_t *k, *v;    // [pages][heads][page_size][D]
    float *ks, *vs;    // [pages][heads][page_size], int8 only
    const int32_t *table;  // [B][W]
    int64_t W;
    int pages, heads, D, shift;  // page_size = 1 << shift
};

// Places of a call's tokens: rows cu[b] .. cu[b + 1] - 1 (cu NULL: row b) are
// sequence b's tokens from position start[b].
struct KvRows {
    const int32_t *start, *cu;
    int64_t T, B;
};

hipError_t launch_kv_append(const KvView &c, bool int8, const KvRows &r, const void *k,
                            const void *v, bool fp32, int64_t ldk, int64_t ldv, hipStream_t st);
hipError_t launch_kv_gather(const KvView &c, bool int8, const KvRows &r, void *k, void *v,
                            bool fp32, hipStream_t st);

// Attention.  cu == NULL: one query per sequence (T = B).
struct KvAttnArgs {
    KvView c;
    bool int8, fp32;     // cache codes; activations
    const void *q;
    int64_t ldq;
    void *out;
    const int32_t *lens, *cu;
    int64_t T, B;
    int hq;              // query heads
    float scale;
    int window, sinks;   // at most 2^30
    void *ws;
};

size_t kv_attn_ws_bytes(int64_t rows, int64_t hq, int64_t heads, int64_t D);
// `path`: the kernel variant taken.
hipError_t launch_kv_attention(const KvAttnArgs &a, const char **path, hipStream_t st);

// Page moves: the cache's arrays as planes of whole pages.
struct KvPlanes {
    uint8_t *k, *v;
    float *ks, *vs;       // NULL: none
    int64_t layers, pages;
    int64_t page_bytes;   // of one K (or V) page
    int64_t scale_bytes;  // of one page of scales (0: none)
};

hipError_t launch_kv_copy_pages(const KvPlanes &dst, const int32_t *dst_ids, const KvPlanes &src,
                                const int32_t *src_ids, int64_t n, hipStream_t st);
hipError_t launch_kv_reserve(int32_t *table, int64_t S, int64_t W, const int32_t *lens,
                             int32_t *refs, int64_t pages, int shift, const int32_t *add,
                             int32_t *ok, int32_t *ws, hipStream_t st);
hipError_t launch_kv_fork(const KvPlanes &c, int shift, int32_t *table, int64_t S, int64_t W,
                          int32_t *lens, int32_t *refs, const int32_t *parents,
                          const int32_t *children, int64_t n, int32_t *ok, int32_t *ws,
                          hipStream_t st);
hipError_t launch_kv_free(int32_t *table, int64_t S, int64_t W, int32_t *lens, int32_t *refs,
                          int64_t pages, const int32_t *slots, int64_t n, hipStream_t st);
hipError_t launch_kv_compact(const KvPlanes &c, const int32_t *table, int64_t S, int64_t W,
                             const int32_t *refs, int32_t *table_out, int32_t *refs_out,
                             int32_t *live, int32_t *ws, hipStream_t st);

}  // namespace w4
