// Dispatch of the attention over the paged key-value cache.
#include "kv_attn.h"

namespace w4 {

size_t kv_attn_ws_bytes(int64_t rows, int64_t hq, int64_t heads, int64_t D) {
    return std::max(kv_decode_ws_bytes(hq, heads, D), kv_prefill_ws_bytes(rows, hq, heads, D));
}

hipError_t launch_kv_attention(const KvAttnArgs &a, const char **path, hipStream_t st) {
    return a.cu ? launch_kv_prefill(a, path, st) : launch_kv_decode(a, path, st);
}

}  // namespace w4
