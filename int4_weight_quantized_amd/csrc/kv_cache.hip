// Paged key-value cache: writing and reading back tokens, and the page moves
// (copy, reserve, fork, free, compact).
#include <algorithm>
#include <type_traits>

#include "kv_common.h"

namespace w4 {

// ------------------------------------------------------------ append, gather
// A group of LPV lanes (8, 16 or 32: head_dim up to 64, 128, 256) handles one
// head's vector of one token, 8 values a lane; blockIdx.y selects K or V.
// Bound by memory: each value is read once and written once (179 MB of prompts, 8
// heads of 128, bf16: 42 us, 4.2 TB/s; a large copy: 4.9; 224 MB of fp32 to int8: 60
// us).  The row's values are loaded before the search for its sequence, and stored past
// the caches.

struct KvPlace {
    int64_t token;   // row of the call, or -1
    int64_t vec;     // (page * heads + head) * page_size + slot, or -1
    int head;
};

template <int LPV>
__device__ __forceinline__ KvPlace kv_place(const KvView &c, const KvRows &r) {
    constexpr int kVecs = 256 / LPV;
    const int64_t n = r.T * c.heads;
    const int64_t first = (int64_t)blockIdx.x * kVecs + threadIdx.x / kWave * (kWave / LPV);
    const int64_t i = (int64_t)blockIdx.x * kVecs + threadIdx.x / LPV;
    KvPlace p{-1, -1, 0};
    int64_t b = 0;
    if (r.cu && first < n) b = find_sequence(r.cu, r.B, first / c.heads);
    if (i >= n) return p;
    p.token = i / c.heads;
    p.head = (int)(i - p.token * c.heads);
    int64_t pos;
    if (r.cu) {
        while (b + 1 < r.B && (int64_t)r.cu[b + 1] <= p.token) ++b;
        if (p.token < r.cu[b] || p.token >= r.cu[b + 1]) return p;
        pos = p.token - r.cu[b];
    } else {
        b = p.token;
        pos = 0;
    }
    const int start = r.start[b];
    if (start < 0) return p;
    pos += start;
    const int page = kv_page(c, c.table + b * c.W, pos);
    if (page >= 0)
        p.vec = (((int64_t)page * c.heads + p.head) << c.shift) + (pos & ((1 << c.shift) - 1));
    return p;
}

template <bool FP32>
__device__ __forceinline__ void load8(const void *x, int64_t at, bool vec, float (&f)[8]) {
    if constexpr (FP32) {
        const float *s = reinterpret_cast<const float *>(x) + at;
        if (vec) {
            const float4 a = *reinterpret_cast<const float4 *>(s);
            const float4 b = *reinterpret_cast<const float4 *>(s + 4);
            f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
            f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = s[j];
        }
    } else {
        const uint16_t *s = reinterpret_cast<const uint16_t *>(x) + at;
        if (vec) {
            const uint4 a = *reinterpret_cast<const uint4 *>(s);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) f[2 * j] = bf16_lo(w[j]), f[2 * j + 1] = bf16_hi(w[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = __uint_as_float((uint32_t)s[j] << 16);
        }
    }
}

// Rounding to the cache's type happens once, here: bf16 half to even, or int8 with
// the scale absmax * fl(1 / 127) of the head's vector (one multiplication, within
// one unit in the last place of the quotient) and codes rne(fl(x / scale)).  A
// vector with a value that is not finite has no int8 form: its scale is NaN.
template <bool INT8, bool FP32, int LPV>
__global__ __launch_bounds__(256) void k_kv_append(KvView c, KvRows r, const void *k,
                                                   const void *v, int64_t ldk, int64_t ldv,
                                                   bool vec) {
    const bool isv = blockIdx.y != 0;
    const int d = threadIdx.x % LPV * 8;
    const int64_t i = (int64_t)blockIdx.x * (256 / LPV) + threadIdx.x / LPV;
    float f[8] = {};
    if (i < r.T * c.heads && d < c.D) {  // (in flight during the search for the place)
        const int64_t token = i / c.heads;
        load8<FP32>(isv ? v : k, token * (isv ? ldv : ldk) + (i - token * c.heads) * c.D + d, vec,
                    f);
    }
    const KvPlace p = kv_place<LPV>(c, r);
    const bool on = p.vec >= 0 && d < c.D;
    uint8_t *pool = isv ? c.v : c.k;
    if constexpr (INT8) {
        // the bits of |x| order as the values do, infinity and NaN above them all
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = LPV / 2; o >= 1; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, kWave));
        if (!on) return;
        const float s = m < 0x7F800000u ? __uint_as_float(m) * (1.0f / 127.0f) : NAN;
        uint32_t w[2] = {};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j / 4] |= (uint32_t)(quant_code(f[j], s, -128.0f, 127.0f) & 0xFF) << (j % 4 * 8);
        *reinterpret_cast<uint2 *>(pool + p.vec * c.D + d) = uint2{w[0], w[1]};
        if (d == 0) (isv ? c.vs : c.ks)[p.vec] = s;
    } else {
        if (!on) return;
        const u32x4 o = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                         pack_bf16(f[6], f[7])};
        __builtin_nontemporal_store(o, reinterpret_cast<u32x4 *>(pool + (p.vec * c.D + d) * 2));
    }
}

template <bool INT8, bool FP32, int LPV>
__global__ __launch_bounds__(256) void k_kv_gather(KvView c, KvRows r, void *k, void *v) {
    const bool isv = blockIdx.y != 0;
    const KvPlace p = kv_place<LPV>(c, r);
    const int d = threadIdx.x % LPV * 8;
    if (p.token < 0 || d >= c.D) return;
    float f[8] = {};
    const uint8_t *pool = isv ? c.v : c.k;
    if (p.vec >= 0) {
        if constexpr (INT8) {
            const uint2 w = *reinterpret_cast<const uint2 *>(pool + p.vec * c.D + d);
            const float s = (isv ? c.vs : c.ks)[p.vec];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f[j] = (float)(int8_t)((j < 4 ? w.x : w.y) >> (j % 4 * 8)) * s;
        } else {
            const uint4 a = *reinterpret_cast<const uint4 *>(pool + (p.vec * c.D + d) * 2);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) f[2 * j] = bf16_lo(w[j]), f[2 * j + 1] = bf16_hi(w[j]);
        }
    }
    const int64_t at = (p.token * c.heads + p.head) * c.D + d;
    if constexpr (FP32) {
        float4 *o = reinterpret_cast<float4 *>(reinterpret_cast<float *>(isv ? v : k) + at);
        o[0] = float4{f[0], f[1], f[2], f[3]};
        o[1] = float4{f[4], f[5], f[6], f[7]};
    } else {
        uint4 o;
        o.x = pack_bf16(f[0], f[1]);
        o.y = pack_bf16(f[2], f[3]);
        o.z = pack_bf16(f[4], f[5]);
        o.w = pack_bf16(f[6], f[7]);
        *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(isv ? v : k) + at) = o;
    }
}

// Calls f with the compile-time lanes per vector / truth value.
template <class F>
static void with_lanes(int D, F f) {
    if (D <= 64)
        f(std::integral_constant<int, 8>{});
    else if (D <= 128)
        f(std::integral_constant<int, 16>{});
    else
        f(std::integral_constant<int, 32>{});
}

template <class F>
static void with_bool(bool b, F f) {
    if (b)
        f(std::true_type{});
    else
        f(std::false_type{});
}

hipError_t launch_kv_append(const KvView &c, bool int8, const KvRows &r, const void *k,
                            const void *v, bool fp32, int64_t ldk, int64_t ldv, hipStream_t st) {
    // 16-byte loads where every row starts on one (head_dim is a multiple of 16)
    const int64_t per = fp32 ? 4 : 8;
    const bool vec = ldk % per == 0 && ldv % per == 0 &&
                     (reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) % 16 == 0;
    with_lanes(c.D, [&](auto lanes) {
        with_bool(int8, [&](auto i8) {
            with_bool(fp32, [&](auto f32) {
                constexpr int L = decltype(lanes)::value;
                const dim3 g((unsigned)((r.T * c.heads + 256 / L - 1) / (256 / L)), 2);
                launch_kv(k_kv_append<decltype(i8)::value, decltype(f32)::value, L>, g, dim3(256),
                          0, st, c, r, k, v, ldk, ldv, vec);
            });
        });
    });
    return hipGetLastError();
}

hipError_t launch_kv_gather(const KvView &c, bool int8, const KvRows &r, void *k, void *v,
                            bool fp32, hipStream_t st) {
    with_lanes(c.D, [&](auto lanes) {
        with_bool(int8, [&](auto i8) {
            with_bool(fp32, [&](auto f32) {
                constexpr int L = decltype(lanes)::value;
                const dim3 g((unsigned)((r.T * c.heads + 256 / L - 1) / (256 / L)), 2);
                launch_kv(k_kv_gather<decltype(i8)::value, decltype(f32)::value, L>, g, dim3(256),
                          0, st, c, r, k, v);
            });
        });
    });
    return hipGetLastError();
}

// ----------------------------------------------------------------- page moves
// Copy of page src[i] to page dst[i] in every plane (K and V of each layer,
// and their scales), i below n or, on the device, below *count.  A workgroup
// copies up to kCopyChunk bytes of one plane's page per step of a grid-stride
// loop, four 16-byte loads a thread in flight, past the caches; bound by memory
// (each byte read once and written once: 3.2 GB in 614 to 629 us, 5.2 TB/s, where a large
// library copy reaches 4.9; a compaction in a loop: 508 us, with 2048 workgroups
// 528, with 65536 500, where 256 forks take 82 us with either of the latter two).
constexpr int64_t kCopyChunk = 32768, kCopyBlocks = 8192;

__device__ __forceinline__ void copy_bytes(uint8_t *d, const uint8_t *s, int bytes) {
    // 4 loads in flight a thread; each byte is used once
    constexpr int kStep = 256 * 16;
    const int at = threadIdx.x * 16;
    int i = at;
    for (; i + 3 * kStep < bytes; i += 4 * kStep) {
        u32x4 x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(s + i + j * kStep));
#pragma unroll
        for (int j = 0; j < 4; ++j)
            __builtin_nontemporal_store(x[j], reinterpret_cast<u32x4 *>(d + i + j * kStep));
    }
    for (; i < bytes; i += kStep)
        __builtin_nontemporal_store(
            __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(s + i)),
            reinterpret_cast<u32x4 *>(d + i));
}

// Units u0, u0 + step, ... of the copies of `pairs` pages.
__device__ __forceinline__ void copy_units(const KvPlanes &D, const int32_t *dst,
                                           const KvPlanes &S, const int32_t *src, int64_t pairs,
                                           int64_t u0, int64_t step) {
    const int64_t chunks = (S.page_bytes + kCopyChunk - 1) / kCopyChunk;
    const int64_t per_layer = 2 * chunks + (S.scale_bytes ? 2 : 0);
    const int64_t per_pair = per_layer * S.layers;
    for (int64_t u = u0; u < pairs * per_pair; u += step) {
        const int64_t i = u / per_pair;
        int64_t x = u - i * per_pair;
        const int from = src[i], to = dst[i];
        if ((uint64_t)(int64_t)from >= (uint64_t)S.pages ||
            (uint64_t)(int64_t)to >= (uint64_t)D.pages)
            continue;
        const int64_t layer = x / per_layer;
        x -= layer * per_layer;
        const int64_t fp = layer * S.pages + from, tp = layer * D.pages + to;
        if (x < 2 * chunks) {
            const bool isv = x >= chunks;
            const int64_t at = (isv ? x - chunks : x) * kCopyChunk;
            copy_bytes((isv ? D.v : D.k) + tp * S.page_bytes + at,
                       (isv ? S.v : S.k) + fp * S.page_bytes + at,
                       (int)min(kCopyChunk, S.page_bytes - at));
        } else {
            const bool isv = x > 2 * chunks;
            for (int64_t at = 0; at < S.scale_bytes; at += kCopyChunk)
                copy_bytes(reinterpret_cast<uint8_t *>(isv ? D.vs : D.ks) + tp * S.scale_bytes + at,
                           reinterpret_cast<const uint8_t *>(isv ? S.vs : S.ks) +
                               fp * S.scale_bytes + at,
                           (int)min(kCopyChunk, S.scale_bytes - at));
        }
    }
}

__global__ __launch_bounds__(256) void k_kv_copy_pages(KvPlanes D, const int32_t *dst, KvPlanes S,
                                                       const int32_t *src, int64_t n) {
    copy_units(D, dst, S, src, n, blockIdx.x, gridDim.x);
}

// Workgroups for the copies of n pages.
static int64_t copy_blocks(const KvPlanes &src, int64_t n) {
    const int64_t chunks = (src.page_bytes + kCopyChunk - 1) / kCopyChunk;
    return std::min<int64_t>(n * src.layers * (2 * chunks + (src.scale_bytes ? 2 : 0)), kCopyBlocks);
}

hipError_t launch_kv_copy_pages(const KvPlanes &dst, const int32_t *dst_ids, const KvPlanes &src,
                                const int32_t *src_ids, int64_t n, hipStream_t st) {
    launch_kv(k_kv_copy_pages, dim3((unsigned)copy_blocks(src, n)), dim3(256), 0, st, dst,
                       dst_ids, src, src_ids, n);
    return hipGetLastError();
}

// ------------------------------------------------- page bookkeeping (one block)
// Reference counts and tables are small next to the pages; one workgroup walks
// them, so that ranks come from prefix sums in index order and every result is
// the same whatever the timing.  Bound by the latency of one step after another (a
// fork's plan 5.5 us at 300 pages and 8.0 at 6000, a compaction's 4.0 at 257 and 6.8
// at 1536, a reservation 4.5 for 64 slots of 8000 pages where none is due and 5.6
// where every slot gets one).
constexpr int kPlan = 1024;

// Inclusive prefix sum over the workgroup; `total` gets the sum of all.
__device__ __forceinline__ int block_scan(int v, int *red, int &total) {
    const int lane = threadIdx.x % kWave, w = threadIdx.x / kWave;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const int t = __shfl_up(v, o, kWave);
        if (lane >= o) v += t;
    }
    if (lane == kWave - 1) red[w] = v;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kPlan / kWave; ++i) {
        const int r = red[i];
        if (i < w) before += r;
        all += r;
    }
    __syncthreads();
    total = all;
    return v + before;
}

// Free pages among refs, counted up to `enough`.
__device__ __forceinline__ int count_free(const int32_t *refs, int64_t pages, int enough,
                                          int *red) {
    int found = 0;
    for (int64_t at = 0; at < pages && found < enough; at += kPlan) {
        const int64_t p = at + threadIdx.x;
        int total;
        block_scan(p < pages && refs[p] == 0 ? 1 : 0, red, total);
        found += total;
    }
    return found;
}

// need[s] pages from entry first[s] on; see w4.h for the rule.
__global__ __launch_bounds__(kPlan) void k_kv_reserve(int32_t *table, int64_t S, int64_t W,
                                                      const int32_t *lens, int32_t *refs,
                                                      int64_t pages, int shift,
                                                      const int32_t *add, int32_t *ok,
                                                      int32_t *upto, int32_t *first) {
    __shared__ int red[kPlan / kWave];
    int sum = 0;
    for (int64_t at = 0; at < S; at += kPlan) {
        const int64_t s = at + threadIdx.x;
        int need = 0, j0 = 0, served = 1;
        if (s < S && add[s] > 0) {
            const int64_t len = lens[s];
            const int64_t end = (len + add[s] + (1 << shift) - 1) >> shift;
            if (len < 0 || end > W) {
                served = 0;
            } else {
                int64_t j = len >> shift;
                while (j < end && table[s * W + j] >= 0) ++j;
                j0 = (int)j;
                need = (int)(end - j);
            }
        }
        int total;
        const int incl = sum + block_scan(need, red, total);
        sum += total;
        if (s < S) {
            upto[s] = incl;
            first[s] = j0;
            ok[s] = served;
        }
    }
    const int nfree = count_free(refs, pages, sum, red);
    // the granted pages: the largest prefix that the free pages cover
    int granted = 0;
    for (int64_t at = 0; at < S; at += kPlan) {
        const int64_t s = at + threadIdx.x;
        int got = 0;
        if (s < S) {
            if (upto[s] <= nfree)
                got = upto[s];
            else if (upto[s] > (s ? upto[s - 1] : 0))
                ok[s] = 0;
        }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) got = max(got, __shfl_xor(got, o, kWave));
        if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = got;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPlan / kWave; ++i) granted = max(granted, red[i]);
        __syncthreads();
    }
    int rank = 0;
    for (int64_t at = 0; at < pages && rank < granted; at += kPlan) {
        const int64_t p = at + threadIdx.x;
        const bool is_free = p < pages && refs[p] == 0;
        int total;
        const int r = rank + block_scan(is_free ? 1 : 0, red, total) - 1;
        rank += total;
        if (is_free && r < granted) {
            int64_t lo = 0, hi = S - 1;  // the slot whose range of ranks holds r
            while (lo < hi) {
                const int64_t mid = (lo + hi) / 2;
                if (upto[mid] > r)
                    hi = mid;
                else
                    lo = mid + 1;
            }
            table[lo * W + first[lo] + (r - (lo ? upto[lo - 1] : 0))] = (int)p;
            refs[p] = 1;
        }
    }
}

hipError_t launch_kv_reserve(int32_t *table, int64_t S, int64_t W, const int32_t *lens,
                             int32_t *refs, int64_t pages, int shift, const int32_t *add,
                             int32_t *ok, int32_t *ws, hipStream_t st) {
    launch_kv(k_kv_reserve, dim3(1), dim3(kPlan), 0, st, table, S, W, lens, refs, pages,
                       shift, add, ok, ws, ws + S);
    return hipGetLastError();
}

// Fork, first step: which forks are granted and their new pages.  Output per
// fork: src / dst page of a partial page's copy (-1: none) and the child's
// length (-1: not granted).  A child named twice goes to the first fork that
// names it: each claims the child's first entry with an atomic minimum that
// the lowest index wins.
__global__ __launch_bounds__(kPlan) void k_kv_fork_plan(int32_t *table, int64_t S, int64_t W,
                                                        int32_t *lens, int32_t *refs,
                                                        int64_t pages, int shift,
                                                        const int32_t *parents,
                                                        const int32_t *children, int64_t n,
                                                        int32_t *ok, int32_t *src, int32_t *dst,
                                                        int32_t *len, int32_t *upto) {
    __shared__ int red[kPlan / kWave];
    for (int64_t i = threadIdx.x; i < n; i += kPlan) {
        const int64_t p = parents[i], c = children[i];
        bool good = p >= 0 && p < S && c >= 0 && c < S;
        if (good) good = lens[c] == 0 && table[c * W] == -1;
        int l = -1, from = -1;
        if (good) {
            l = lens[p];
            good = l >= 0 && ((int64_t)l + (1 << shift) - 1) >> shift <= W;
            if (good && (l & ((1 << shift) - 1))) {
                from = table[p * W + (l >> shift)];
                good = from >= 0 && from < pages;
            }
        }
        ok[i] = good;
        len[i] = good ? l : -1;
        src[i] = good ? from : -1;
        dst[i] = -1;
    }
    __syncthreads();
    for (int64_t i = threadIdx.x; i < n; i += kPlan)
        if (ok[i]) atomicMin(&table[(int64_t)children[i] * W], (int)(i - n - 1));
    __syncthreads();
    int sum = 0;
    for (int64_t at = 0; at < n; at += kPlan) {
        const int64_t i = at + threadIdx.x;
        int need = 0;
        if (i < n && ok[i]) {
            const int claim = __hip_atomic_load(&table[(int64_t)children[i] * W],
                                                __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (claim != (int)(i - n - 1)) {
                ok[i] = 0;
                len[i] = -1;
                src[i] = -1;
            } else {
                need = src[i] >= 0;
            }
        }
        int total;
        const int incl = sum + block_scan(need, red, total);
        sum += total;
        if (i < n) upto[i] = incl;
    }
    const int nfree = count_free(refs, pages, sum, red);
    for (int64_t i = threadIdx.x; i < n; i += kPlan) {
        if (!ok[i]) continue;
        if (upto[i] > nfree) {  // (a fork that needs no page is denied behind one that is)
            table[(int64_t)children[i] * W] = -1;
            ok[i] = 0;
            len[i] = -1;
            src[i] = -1;
        } else {
            lens[children[i]] = len[i];
        }
    }
    // deal the free pages: the fork with rank r is the first with upto > r
    const int granted = min(sum, nfree);
    int rank = 0;
    for (int64_t at = 0; at < pages && rank < granted; at += kPlan) {
        const int64_t p = at + threadIdx.x;
        const bool is_free = p < pages && refs[p] == 0;
        int total;
        const int r = rank + block_scan(is_free ? 1 : 0, red, total) - 1;
        rank += total;
        if (is_free && r < granted) {
            int64_t lo = 0, hi = n - 1;
            while (lo < hi) {
                const int64_t mid = (lo + hi) / 2;
                if (upto[mid] > r)
                    hi = mid;
                else
                    lo = mid + 1;
            }
            dst[lo] = (int)p;
            refs[p] = 1;
        }
    }
}

// Fork, second step: workgroups 0 .. n - 1 write the children's rows and count the
// shared pages, the others copy the partial pages.
__global__ __launch_bounds__(256) void k_kv_fork_apply(KvPlanes c, int32_t *table, int64_t W,
                                                       int32_t *refs, int shift,
                                                       const int32_t *parents,
                                                       const int32_t *children, int64_t n,
                                                       const int32_t *src, const int32_t *dst,
                                                       const int32_t *len) {
    const int64_t i = blockIdx.x;
    if (i >= n) {
        copy_units(c, dst, c, src, n, i - n, gridDim.x - n);
        return;
    }
    const int l = len[i];
    if (l < 0) return;
    const int64_t full = l >> shift;
    const int32_t *from = table + (int64_t)parents[i] * W;
    int32_t *to = table + (int64_t)children[i] * W;
    for (int64_t j = threadIdx.x; j < W; j += 256) {
        int p = -1;
        if (j < full) {
            p = from[j];
            if (p >= 0 && p < c.pages) atomicAdd(&refs[p], 1);
        } else if (j == full) {
            p = dst[i];
        }
        to[j] = p;
    }
}

hipError_t launch_kv_fork(const KvPlanes &c, int shift, int32_t *table, int64_t S, int64_t W,
                          int32_t *lens, int32_t *refs, const int32_t *parents,
                          const int32_t *children, int64_t n, int32_t *ok, int32_t *ws,
                          hipStream_t st) {
    int32_t *src = ws, *dst = ws + n, *len = ws + 2 * n, *upto = ws + 3 * n;
    launch_kv(k_kv_fork_plan, dim3(1), dim3(kPlan), 0, st, table, S, W, lens, refs,
                       c.pages, shift, parents, children, n, ok, src, dst, len, upto);
    hipLaunchKernelGGL(k_kv_fork_apply, dim3((unsigned)(n + copy_blocks(c, n))), dim3(256), 0, st,
                       c, table, W, refs, shift, parents, children, n, src, dst, len);
    return hipGetLastError();
}

// Every entry is taken out of its row by an atomic exchange, so that a slot
// named twice gives its pages back once.
__global__ __launch_bounds__(256) void k_kv_free(int32_t *table, int64_t S, int64_t W,
                                                 int32_t *lens, int32_t *refs, int64_t pages,
                                                 const int32_t *slots, int64_t n) {
    const int64_t s = slots[blockIdx.x];
    if (s < 0 || s >= S) return;
    for (int64_t j = threadIdx.x; j < W; j += 256) {
        const int p = atomicExch(&table[s * W + j], -1);
        if (p >= 0 && p < pages) atomicSub(&refs[p], 1);
    }
    if (threadIdx.x == 0) lens[s] = 0;
}

hipError_t launch_kv_free(int32_t *table, int64_t S, int64_t W, int32_t *lens, int32_t *refs,
                          int64_t pages, const int32_t *slots, int64_t n, hipStream_t st) {
    launch_kv(k_kv_free, dim3((unsigned)n), dim3(256), 0, st, table, S, W, lens, refs,
                       pages, slots, n);
    return hipGetLastError();
}

// Compaction, first step: the moves (src, dst: `moves` of them) and the new
// reference counts.
__global__ __launch_bounds__(kPlan) void k_kv_compact_plan(const int32_t *refs, int32_t *refs_out,
                                                           int64_t pages, int32_t *live,
                                                           int32_t *moves, int32_t *src,
                                                           int32_t *dst) {
    __shared__ int red[kPlan / kWave];
    int n = 0;
    for (int64_t at = 0; at < pages; at += kPlan) {
        const int64_t p = at + threadIdx.x;
        int total;
        block_scan(p < pages && refs[p] > 0 ? 1 : 0, red, total);
        n += total;
    }
    int holes = 0, movers = 0;
    for (int64_t at = 0; at < pages; at += kPlan) {
        const int64_t p = at + threadIdx.x;
        const bool is_live = p < pages && refs[p] > 0;
        const bool hole = p < n && !is_live, mover = p >= n && is_live;
        int nh, nm;
        const int h = holes + block_scan(hole ? 1 : 0, red, nh) - 1;
        const int m = movers + block_scan(mover ? 1 : 0, red, nm) - 1;
        holes += nh;
        movers += nm;
        if (hole) dst[h] = (int)p;
        if (mover) src[m] = (int)p;
        if (p < pages && !hole && !mover) refs_out[p] = refs[p];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < movers; i += kPlan) {
        const int from = src[i], to = dst[i];
        const int r = refs[from];
        refs_out[to] = r;
        refs_out[from] = 0;
    }
    if (threadIdx.x == 0) {
        live[0] = n;
        moves[0] = movers;
    }
}

// Compaction, second step: the first `tables` workgroups rename the table's
// entries (a moved page's new place is found in the sorted list of moves), the
// others copy the pages.
__global__ __launch_bounds__(256) void k_kv_compact_apply(KvPlanes c, const int32_t *table,
                                                          int32_t *table_out, int64_t entries,
                                                          int64_t tables, const int32_t *live,
                                                          const int32_t *moves,
                                                          const int32_t *src,
                                                          const int32_t *dst) {
    const int n = moves[0];
    if (blockIdx.x >= tables) {
        copy_units(c, dst, c, src, n, blockIdx.x - tables, gridDim.x - tables);
        return;
    }
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= entries) return;
    int p = table[i];
    if (p < 0 || p >= c.pages) {
        p = -1;
    } else if (p >= live[0]) {
        int lo = 0, hi = n;
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (src[mid] < p)
                lo = mid + 1;
            else
                hi = mid;
        }
        if (lo < n && src[lo] == p) p = dst[lo];
    }
    table_out[i] = p;
}

hipError_t launch_kv_compact(const KvPlanes &c, const int32_t *table, int64_t S, int64_t W,
                             const int32_t *refs, int32_t *table_out, int32_t *refs_out,
                             int32_t *live, int32_t *ws, hipStream_t st) {
    int32_t *moves = ws, *src = ws + 4, *dst = src + c.pages;
    launch_kv(k_kv_compact_plan, dim3(1), dim3(kPlan), 0, st, refs, refs_out, c.pages,
                       live, moves, src, dst);
    // at most half of the pages move (a move needs a live page and a hole)
    const int64_t tables = (S * W + 255) / 256;
    const int64_t blocks = tables + copy_blocks(c, std::max<int64_t>(c.pages / 2, 1));
    hipLaunchKernelGGL(k_kv_compact_apply, dim3((unsigned)blocks), dim3(256), 0, st, c, table,
                       table_out, S * W, tables, live, moves, src, dst);
    return hipGetLastError();
}

}  // namespace w4
