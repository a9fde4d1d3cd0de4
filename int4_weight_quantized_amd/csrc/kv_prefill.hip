// Attention of prompts (or chunks of them) over the paged key-value cache.
//
// Online softmax over tiles of 64 tokens: for every tile S = Q K^T, a running
// maximum m and sum l, O = O e^(m_old - m) + P V.  A workgroup has 128 query
// rows of one sequence and cache head, a wave 32 of them; a row is a (token,
// query head) pair, so the G = q_heads / heads query heads that share a cache
// head share its tiles, and causal tiles are skipped for 128 / G tokens at a
// time.
//
// Both products are taken transposed (S^T = K Q^T, O^T = V^T P^T) with
// v_mfma_f32_32x32x16_bf16: a lane holds one query row throughout, so that
// maxima, sums and rescaling need one exchange between two lanes, and the
// accumulators of S^T are the B operand of the second product as they stand
// (the order of tokens inside its depth is free; V is read to match).
//
// K and V tiles lie in LDS row by row, 16-byte chunks XOR-swizzled so that the
// reads cover all banks evenly; V^T comes out of its rows by the transposing
// read ds_read_b64_tr_b16 (16 lanes read 4 rows of 16 values and get a column's
// 4 each).  A bf16 cache goes to LDS directly (no registers, the swizzle is in
// each lane's global address), int8 codes through registers, where they become
// bf16 (exact); their scales multiply the scores and the softmax weights (a
// workgroup that meets a scale of V outside 2^-110 to 2^50 takes its rows token by
// token instead, see plain_row).  Two
// LDS buffers, the next tile's loads in flight during this one's products, one
// barrier a tile; a wave loads the 16 tokens of one quarter, so that it needs
// one page.
//
// The maximum is only moved when a score passes it by 8 (in units of log 2):
// weights up to 2^8 lose nothing in bf16 or fp32, and the 64 to 128
// accumulators are rarely rescaled.
//
// Rounding: bf16 activations have their softmax weights rounded to bf16 once (two
// terms: 318 us where one took 265, int8); fp32 ones are three bf16 terms, q and
// weights alike, so that products keep 24 bits.  Sums and statistics are fp32.
//
// 8192 causal tokens, 32 / 8 heads of 128, bf16: 527 to 557 us by card, 0.99 to 1.04
// PFLOP/s (large library products in bf16: 1.21 to 1.36).  The MFMAs are busy 49% of
// 1.08 million cycles.  A schedule with the next tile's scores beside this one's
// exponentials was no faster (557 us where 559 without) and spilled registers for int8.
// fp32 activations, three products for one: 1472 us.
// int8 adds the conversion of codes and the scales: 277 to 289 us for ragged prompts up
// to 8000 with a window of 1024, 16 / 4 heads of 128.  256 rows a workgroup share that
// work among more rows, but took 274 us where 128 took 265 (both before the weights'
// sum was taken from their rounded values).
#include "kv_attn.h"

namespace w4 {

namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kRows = 128, kTile = 64, kThreads = 256;
constexpr float kSlack = 8.0f;
// int8: weights are held 2^kShift times as large, so that the scales of V that the
// products take reach from 2^-110 to 2^50 (values of an ordinary model lie between 2^-30
// and 2^20): a weight of 2^-46 times the least scale is still a normal number, and
// 2^8 times the largest one and its reciprocal are far from the other end.
constexpr float kShift = 30.0f, kScaleMin = 0x1p-110f, kScaleMax = 0x1p50f;

__device__ __forceinline__ v16f mfma32(uint4 a, uint4 b, v16f c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a),
                                                   __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// Swizzles: what the index of a token's 16-byte chunk is XORed with.  K is read
// 16 rows of one chunk at a time, V 4 rows of 4 chunks (half a transposing
// read); a row of 64 values is half of the banks.
template <int DP>
__device__ __forceinline__ int k_swizzle(int t) {
    return DP == 64 ? (t >> 1) & 7 : t & 15;
}
template <int DP>
__device__ __forceinline__ int v_swizzle(int t) {
    return DP == 64 ? ((t >> 1) & 1) * 4 : (t & 3) * 4;
}

// Tile index of the first tile of sequence b: the sequences' tiles lie in
// disjoint ranges (a sequence of n rows has at most floor(n / 128) + 1 more).
__device__ __forceinline__ int64_t first_tile(const KvAttnArgs &a, int G, int64_t b) {
    return (int64_t)a.cu[b] * G / kRows + b;
}

// The last sequence whose first tile is at or before `idx` (wave-uniform).
__device__ __forceinline__ int64_t find_tile(const KvAttnArgs &a, int G, int64_t idx) {
    const int lane = threadIdx.x % kWave;
    int64_t lo = 0, n = a.B - 1;
    while (n > 0) {
        const int64_t step = (n + 63) / 64;
        const int64_t off = (int64_t)(lane + 1) * step;
        const bool below = off <= n && first_tile(a, G, lo + off) <= idx;
        const int64_t c = __popcll(__ballot(below));
        lo += c * step;
        n = min(step - 1, n - c * step);
    }
    return lo;
}

// c + the products of two packed bf16 pairs (`one`: both 1).
constexpr uint32_t one = 0x3F803F80u;
__device__ __forceinline__ float dot_pair(uint32_t w, uint32_t x, float c) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w),
                                           __builtin_bit_cast(bf16x2, x), c, false);
}

// Parts that the tiles of a workgroup's rows are split over.
constexpr int kMaxParts = 16;

// Where a row's result goes: to its place in the output, or, where the tiles of a
// row go to several workgroups, as the unnormalized part of this one.
struct RowOut {
    int64_t row;   // token * q_heads + head
    int part, parts;
    __device__ float *sums(const KvAttnArgs &a) const {  // D sums, m, l
        return reinterpret_cast<float *>(a.ws) + (row * parts + part) * (a.c.D + 4);
    }
};

// One query row without the matrix cores, token by token, so that a token the
// row does not see takes no part at all and a value is code * scale whatever the
// scale: for workgroups whose edge tiles hold infinities or NaN in V (the products
// of a tile would carry them to every row as 0 * inf), or whose tiles hold scales of
// V outside kScaleMin to kScaleMax.  About 12 us a row and tile, for what should
// not be there at all.  The whole workgroup, `buf` 512 floats of LDS; tile_token(i) is
// the first token of tile i, i from i0 to i1 - 1.
template <bool INT8, bool FP32, class F>
__device__ void plain_row(const KvAttnArgs &a, const int32_t *table, int64_t token, int h, int kvh,
                          int pos, F tile_token, int i0, int i1, RowOut out, float *buf) {
    float *q = buf, *p = buf + 256;
    int64_t *vecs = reinterpret_cast<int64_t *>(p + 128);  // of the tile's tokens, -1: not seen
    const int tid = threadIdx.x, D = a.c.D;
    const int low = a.window ? pos - a.window + 1 : 0;
    __syncthreads();
    if (tid < D) {
        const int64_t at = token * a.ldq + (int64_t)h * D + tid;
        q[tid] = FP32 ? reinterpret_cast<const float *>(a.q)[at]
                      : bf16_lo(reinterpret_cast<const uint16_t *>(a.q)[at]);
    }
    auto value = [&](const uint8_t *pool, const float *scales, int64_t vec, int d) {
        if constexpr (INT8)
            return (float)(int8_t)pool[vec * D + d] * scales[vec];
        else
            return bf16_lo(reinterpret_cast<const uint16_t *>(pool)[vec * D + d]);
    };
    auto key8 = [&](int64_t vec, int d, float (&k)[8]) {
        if constexpr (INT8) {
            const uint2 w = *reinterpret_cast<const uint2 *>(a.c.k + vec * D + d);
            const float s = a.c.ks[vec];
#pragma unroll
            for (int j = 0; j < 8; ++j) k[j] = (float)(int8_t)((j < 4 ? w.x : w.y) >> (j % 4 * 8)) * s;
        } else {
            const uint4 w = *reinterpret_cast<const uint4 *>(a.c.k + (vec * D + d) * 2);
            const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) k[2 * j] = bf16_lo(v[j]), k[2 * j + 1] = bf16_hi(v[j]);
        }
    };
    auto vector = [&](int t) {
        const int pg = kv_page(a.c, table, t);
        return pg < 0 ? (int64_t)-1 : kv_vector(a.c, pg, kvh, t);
    };
    float m = -INFINITY, l = 0.0f, o = 0.0f;
    for (int i = i0; i < i1; ++i) {
        __syncthreads();
        const int t0 = tile_token(i), t = t0 + tid;
        if (tid < kTile) {
            const bool see = t <= pos && (t >= low || t < a.sinks);
            const int64_t vec = see ? vector(t) : -1;
            float s = -INFINITY;
            if (vec >= 0) {
                float x = 0.0f;
#pragma unroll 1
                for (int d = 0; d < D; d += 8) {
                    float k[8];
                    key8(vec, d, k);
#pragma unroll
                    for (int j = 0; j < 8; ++j) x = __builtin_fmaf(q[d + j], k[j], x);
                }
                s = x * a.scale * 1.44269504088896340736f;
            }
            const float mn = fmaxf(m, wave_max(s));
            vecs[tid] = vec;
            p[tid] = vec >= 0 ? __builtin_amdgcn_exp2f(s - mn) : 0.0f;
            if (tid == 0) p[kTile] = mn;
        }
        __syncthreads();
        const float mn = p[kTile];
        const float alpha = mn == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
        m = mn;
        l *= alpha;
        o *= alpha;
#pragma unroll 4
        for (int j = 0; j < kTile; ++j) {
            const int64_t vj = vecs[j];
            l += p[j];
            if (tid < D) {
                const float v = value(a.c.v, a.c.vs, max(vj, (int64_t)0), tid);
                o = __builtin_fmaf(p[j], vj >= 0 ? v : 0.0f, o);
            }
        }
    }
    if (out.parts > 1) {
        float *to = out.sums(a);
        if (tid < D) to[tid] = o;
        if (tid == 0) to[D] = m, to[D + 1] = l;
    } else if (tid < D) {
        const float y = l == 0.0f ? 0.0f : o / l;
        if constexpr (FP32)
            reinterpret_cast<float *>(a.out)[out.row * D + tid] = y;
        else
            reinterpret_cast<__bf16 *>(a.out)[out.row * D + tid] = (__bf16)y;
    }
}

}  // namespace

template <int DP, bool INT8, bool FP32>
__global__ __launch_bounds__(kThreads, DP <= 128 && !FP32 ? 2 : 1) void k_kv_prefill(KvAttnArgs a,
                                                                                          int parts) {
    constexpr int kSteps = DP / 16, kDt = DP / 32, kQ = FP32 ? 3 : 1, kP = kQ;
    constexpr int kPitch = DP * 2, kCh = DP / 8;  // an LDS row: bytes, 16-byte chunks
    constexpr int kVTile = kTile * kPitch, kBuf = 2 * kVTile;
    constexpr int kCode = DP / 16;                // 16-byte chunks of a row of codes
    constexpr int kLoads = INT8 ? DP / 64 : DP / 32;  // loads of 16 rows by a wave
    extern __shared__ __align__(16) uint8_t lds[];
    __shared__ float sks[2][kTile], svs[2][kTile];
    __shared__ __align__(8) uint16_t inv_hi[2][kTile], inv_lo[2][kTile];  // 1 / svs, two bf16 terms
    __shared__ int odd;  // whether a tile has values or scales of V that the products cannot take

    const int tid = threadIdx.x, lane = tid % kWave, half = lane / 32, col = lane % 32;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int D = a.c.D, G = a.hq / a.c.heads;
    const int kvh = (int)(blockIdx.x % a.c.heads), part = blockIdx.y;
    const int64_t idx = (int64_t)gridDim.x / a.c.heads - 1 - blockIdx.x / a.c.heads;
    const int64_t b = find_tile(a, G, idx);
    const int64_t c0 = a.cu[b];
    const int64_t nq = (int64_t)a.cu[b + 1] - c0;
    const int64_t row0 = (idx - first_tile(a, G, b)) * kRows;
    // (rows before the first offset, and offsets that fall or pass T, are no work)
    if (c0 < 0 || nq <= 0 || c0 + nq > a.T || row0 < 0 || row0 >= nq * G) return;

    // this lane's query row
    const int rows = (int)min(nq * G - row0, (int64_t)kRows);
    const int r = min(wave * 32 + col, rows - 1);
    const bool on = wave * 32 + col < rows;
    const int tok = (int)((row0 + r) / G);
    const int head = kvh * G + (int)(row0 + r - (int64_t)tok * G);
    const int len = kv_length(a, b);
    const int pos = on ? len - (int)nq + tok : -1;
    const int low = a.window ? pos - a.window + 1 : 0;

    // positions of the workgroup's rows, and the tokens that any of them sees
    const int pos0 = len - (int)nq + (int)(row0 / G);
    const int pos1 = len - (int)nq + (int)((row0 + rows - 1) / G);
    const int low0 = a.window ? max(pos0 - a.window + 1, 0) : 0;
    const int low1 = a.window ? max(pos1 - a.window + 1, 0) : 0;
    const int lo_tile = low0 / kTile;
    const int sink_tiles = min((a.sinks + kTile - 1) / kTile, lo_tile);
    const int tiles = pos1 < 0 ? 0 : sink_tiles + pos1 / kTile + 1 - lo_tile;
    const int32_t *table = a.c.table + b * a.c.W;
    // this workgroup's share of the tiles
    const int i0 = (int)((int64_t)tiles * part / parts);
    const int i1 = (int)((int64_t)tiles * (part + 1) / parts);

    // scores in units of log 2 are sc times S; a scale below zero turns q's
    // signs, one of zero clears q, so that sc > 0 and the maximum of S serves
    const float sc = a.scale == 0.0f ? 1.0f : fabsf(a.scale) * 1.44269504088896340736f;
    const uint32_t q_and = a.scale == 0.0f ? 0u : ~0u, q_xor = a.scale < 0.0f ? 0x80008000u : 0u;

    // q stays in registers as the B operand, but for the three terms of 256 dims
    // (192 registers beside 128 of O): those are read and split for every tile
    constexpr bool kKeep = !(FP32 && DP == 256);
    const int64_t q_at = (c0 + tok) * a.ldq + head * D + half * 8;
    uint4 q[kQ][kKeep ? kSteps : 1];
    auto load_q = [&](int j, int to) {
        load_query<FP32>(a.q, q_at + j * 16, on && j * 16 + half * 8 < D, q, to);
#pragma unroll
        for (int u = 0; u < kQ; ++u) {
            uint4 &w = q[u][to];
            w = uint4{(w.x & q_and) ^ q_xor, (w.y & q_and) ^ q_xor, (w.z & q_and) ^ q_xor,
                      (w.w & q_and) ^ q_xor};
        }
    };
    if constexpr (kKeep)
#pragma unroll
        for (int j = 0; j < kSteps; ++j) load_q(j, j);

    auto tile_token = [&](int i) {
        return kTile * (i < sink_tiles ? i : i - sink_tiles + lo_tile);
    };
    // pages of the next 16 tiles, one lane for each 16 tokens
    int base = 0, pages = -1;
    uint64_t gone = 0;  // lanes without a page
    auto look_up = [&](int i) {
        const int ii = i + lane / 4;
        base = i;
        pages = ii < i1 ? kv_page(a.c, table, tile_token(ii) + lane % 4 * 16) : -1;
        gone = __ballot(pages < 0);
    };
    auto gone_of = [&](int i) { return (int)(gone >> (4 * (i - base))) & 15; };
    // whether some row does not see some token of the tile
    auto at_edge = [&](int t0, int none) {
        return t0 + kTile - 1 > pos0 || (a.window && t0 < low1 && t0 + kTile > a.sinks) ||
               none != 0;
    };

    // Lane offsets of the loads: chunk (lane % chunks) of LDS row (lane / chunks)
    // holds the token's chunk at that place XOR the row's swizzle.
    constexpr int kRowsPer = INT8 ? 64 / kCode : 64 / kCh;  // rows of a load
    u32x4 stage[INT8 ? 2 * kLoads : 1];
    float ks = 0.0f, vs = 0.0f;
    auto load = [&](int i, int buf) {
        const int t0 = tile_token(i);
        const int pg = __builtin_amdgcn_readlane(pages, 4 * (i - base) + wave);
        const int64_t vec = kv_vector(a.c, max(pg, 0), kvh, t0 + 16 * wave);
        if constexpr (INT8) {
            const int ch = lane % kCode * 16;
            const uint32_t off = lane / kCode * D + (ch < D ? ch : 0);
            const uint8_t *kp = a.c.k + vec * D, *vp = a.c.v + vec * D;
#pragma unroll
            for (int j = 0; j < kLoads; ++j, kp += kRowsPer * D, vp += kRowsPer * D) {
                stage[j] = *reinterpret_cast<const u32x4 *>(kp + off);
                stage[kLoads + j] = *reinterpret_cast<const u32x4 *>(vp + off);
            }
            ks = a.c.ks[vec + lane % 16];
            vs = a.c.vs[vec + lane % 16];
        } else {
            const v4i kd = buffer_desc(a.c.k + vec * D * 2, 16 * D * 2);
            const v4i vd = buffer_desc(a.c.v + vec * D * 2, 16 * D * 2);
            const uint32_t to = lds_addr(lds) + buf * kBuf + wave * 16 * kPitch;
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int t = j * kRowsPer + lane / kCh;  // of the quarter's 16
                const int kc = ((lane % kCh) ^ k_swizzle<DP>(t)) * 8;
                const int vc = ((lane % kCh) ^ v_swizzle<DP>(t)) * 8;
                dma16(kd, to + j * 1024, (t * D + (kc < D ? kc : 0)) * 2, 0);
                dma16(vd, to + kVTile + j * 1024, (t * D + (vc < D ? vc : 0)) * 2, 0);
            }
        }
    };
    // The tile's last steps before its barrier, by the wave that loaded a quarter.
    auto finish = [&](int i, int buf, bool edge) {
        uint8_t *kb = lds + buf * kBuf + wave * 16 * kPitch, *vb = kb + kVTile;
        if constexpr (INT8) {
            // the sum of bf16 weights divides the scales out again: a scale of zero is
            // taken as codes of zero
            const uint64_t zero = FP32 ? 0 : __ballot(vs == 0.0f);  // (lane % 16: the token)
            if (zero) {
#pragma unroll
                for (int j = 0; j < kLoads; ++j)
                    if (zero >> (j * kRowsPer + lane / kCode) & 1) stage[kLoads + j] = u32x4{};
            }
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int t = j * kRowsPer + lane / kCode, ch = lane % kCode * 2;
                const uint4 k = __builtin_bit_cast(uint4, stage[j]);
                const uint4 v = __builtin_bit_cast(uint4, stage[kLoads + j]);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    *reinterpret_cast<uint4 *>(
                        kb + t * kPitch + (((ch + x) ^ k_swizzle<DP>(t)) << 4)) = codes8(k, x);
                    *reinterpret_cast<uint4 *>(
                        vb + t * kPitch + (((ch + x) ^ v_swizzle<DP>(t)) << 4)) = codes8(v, x);
                }
            }
            if (lane < 16) {
                const int at = wave * 16 + lane, t = tile_token(i) + at;
                sks[buf][at] = ks;
                const bool fits = fabsf(vs) >= kScaleMin && fabsf(vs) <= kScaleMax;
                const bool finite = fabsf(vs) < INFINITY;
                // (far off, or not finite for some rows only: plain_row takes what a row
                // sees as it is.  An unseen token's weight of zero stays zero; what is not
                // finite for all rows reaches all of them)
                if (!fits && vs != 0.0f && (edge || finite) && t <= pos1 &&
                    (t >= low0 || t < a.sinks) && !(gone_of(i) >> wave & 1))
                    odd = 1;
                const float v = fits || (FP32 && vs == 0.0f) || !(edge || finite) ? vs : 1.0f;
                svs[buf][at] = v;
                if constexpr (!FP32) {
                    const float inv = 1.0f / v;
                    const uint32_t hi = pack_bf16(inv, 0.0f);
                    inv_hi[buf][at] = (uint16_t)hi;
                    inv_lo[buf][at] = (uint16_t)pack_bf16(inv - bf16_lo(hi), 0.0f);
                }
            }
        } else {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            if (edge) {
                // V of tokens that no row sees may be anything: clear it; what some
                // rows see and others do not must be finite for the product with a
                // weight of zero: note where it is not
                const int t = tile_token(i) + 16 * wave + lane / 4;
                const bool seen = t <= pos1 && (t >= low0 || t < a.sinks) &&
                                  !(gone_of(i) >> wave & 1);
                bool inf = false;
#pragma unroll 1
                for (int ch = lane % 4; ch < kCh; ch += 4) {
                    u32x4 *p = reinterpret_cast<u32x4 *>(vb + lane / 4 * kPitch + ch * 16);
                    const u32x4 x = *p;
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        inf |= (x[w] & 0x7F80u) == 0x7F80u || (x[w] & 0x7F800000u) == 0x7F800000u;
                    if (!seen) *p = u32x4{0, 0, 0, 0};
                }
                if (seen && inf) odd = 1;
            }
        }
    };

    if (tid == 0) odd = 0;
    __syncthreads();
    v16f o[kDt] = {};
    float m = -INFINITY, l = 0.0f;
    bool edge = false;
    int none = 0;
    if (i0 < i1) {
        look_up(i0);
        none = gone_of(i0);
        edge = at_edge(tile_token(i0), none);
        load(i0, i0 & 1);
        finish(i0, i0 & 1, edge);
    }
    __syncthreads();
    // lane addresses in a tile: K's chunk `half` of row col, V's chunk of the
    // first rows of a transposing read (see the top)
    const int k_lane = col * kPitch, k_x = (half ^ k_swizzle<DP>(col)) << 4;
    const int v_row = half * 4 + lane % 16 / 4;
    const int v_lane = v_row * kPitch + (lane & 1) * 8;
    const int v_x = ((lane / 16 % 2 * 2 + lane % 4 / 2) ^ v_swizzle<DP>(v_row)) << 4;
    for (int i = i0; i < i1; ++i) {
        const int buf = i & 1;
        const int t0 = tile_token(i);
        const bool more = i + 1 < i1;
        bool next_edge = false;
        int next_none = 0;
        if (more) {
            if (i + 1 - base >= 16) look_up(i + 1);
            next_none = gone_of(i + 1);
            next_edge = at_edge(tile_token(i + 1), next_none);
            load(i + 1, buf ^ 1);
        }
        const uint8_t *kb = lds + buf * kBuf + k_lane;
        const uint32_t vb = lds_addr(lds) + buf * kBuf + kVTile + v_lane;
        // fragments are read a step ahead of their products (more measured the same)
        constexpr int kDeep = 1;
        v16f s[2] = {};
        uint4 kf[kDeep + 1][2];
        auto read_k = [&](int j) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
                kf[j % (kDeep + 1)][t] =
                    *reinterpret_cast<const uint4 *>(kb + t * 32 * kPitch + (k_x ^ (j * 32)));
        };
#pragma unroll
        for (int j = 0; j < kDeep; ++j) read_k(j);
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            if (j + kDeep < kSteps) read_k(j + kDeep);
            if constexpr (!kKeep) load_q(j, 0);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int u = kQ - 1; u >= 0; --u)
                    s[t] = mfma32(kf[j % (kDeep + 1)][t], q[u][kKeep ? j : 0], s[t]);
        }
        // token of register r: 32 t + 8 (r / 4) + 4 half + r % 4
        if constexpr (INT8) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r4 = 0; r4 < 4; ++r4) {
                    const v4f x =
                        *reinterpret_cast<const v4f *>(&sks[buf][32 * t + 8 * r4 + 4 * half]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[t][4 * r4 + e] *= x[e];
                }
        }
        if (edge) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int tj = t0 + 32 * t + 8 * (r / 4) + 4 * half + r % 4;
                    const bool see = (tj <= pos) & ((tj >= low) | (tj < a.sinks)) &
                                     !(none >> (2 * t + r / 8) & 1);
                    s[t][r] = see ? s[t][r] : -INFINITY;
                }
        }
        // (the other wave of the SIMD is in its products by then: apart in phase, the
        // two share the matrix cores and the VALU better)
        __builtin_amdgcn_s_setprio(1);
        float mt = s[0][0];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) mt = fmaxf(mt, s[t][r]);
        mt *= sc;
        if (__any(mt > m + kSlack)) {
            // (the row's other half is asked only here)
            const float mn = fmaxf(m, fmaxf(mt, __shfl_xor(mt, 32, kWave)));
            const float alpha = m == mn ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= alpha;
#pragma unroll
            for (int d = 0; d < kDt; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[d][r] *= alpha;
        }
        const float mu = m == -INFINITY ? 0.0f : INT8 ? kShift - m : -m;
        constexpr int kAheadV = 1;
        constexpr int kVMask = 0x2 | 0x4 | 0x400;  // VALU, SALU and transcendentals may pass
        uint4 vf[kAheadV + 1];
        auto read_v = [&](int n) {
            const uint32_t at = vb + n / kDt * 16 * kPitch + (v_x ^ (n % kDt * 64));
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)at);
            const s16x4 hi =
                __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(at + 8 * kPitch));
            const uint2 x = __builtin_bit_cast(uint2, lo), y = __builtin_bit_cast(uint2, hi);
            vf[n % (kAheadV + 1)] = uint4{x.x, x.y, y.x, y.y};
        };
#pragma unroll
        for (int n = 0; n < kAheadV; ++n) read_v(n);
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) {  // 16 tokens: registers 8 (i4 % 2) ... of half i4 / 2
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f[j] = __builtin_amdgcn_exp2f(
                    __builtin_fmaf(s[i4 / 2][8 * (i4 % 2) + j], sc, mu));
            if constexpr (FP32) {
#pragma unroll
                for (int j = 0; j < 8; ++j) l += f[j];
            }
            if constexpr (INT8) {
#pragma unroll
                for (int j4 = 0; j4 < 2; ++j4) {
                    const v4f x = *reinterpret_cast<const v4f *>(
                        &svs[buf][16 * i4 + 8 * j4 + 4 * half]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[4 * j4 + e] *= x[e];
                }
            }
            uint4 p[kP];
            split_bf16<kP>(f, p);
            // the sum of the weights as the product takes them, rounded (and their
            // scales divided out): what rounding does to a weight that outweighs the
            // others cancels in O / l
            if constexpr (!FP32) {
                const uint32_t w[4] = {p[0].x, p[0].y, p[0].z, p[0].w};
#pragma unroll
                for (int j4 = 0; j4 < 2; ++j4) {
                    if constexpr (INT8) {
                        const int at = 16 * i4 + 8 * j4 + 4 * half;
                        const uint2 h = *reinterpret_cast<const uint2 *>(&inv_hi[buf][at]);
                        const uint2 x = *reinterpret_cast<const uint2 *>(&inv_lo[buf][at]);
                        l = dot_pair(w[2 * j4], x.x, l);
                        l = dot_pair(w[2 * j4 + 1], x.y, l);
                        l = dot_pair(w[2 * j4], h.x, l);
                        l = dot_pair(w[2 * j4 + 1], h.y, l);
                    } else {
                        l = dot_pair(w[2 * j4], one, l);
                        l = dot_pair(w[2 * j4 + 1], one, l);
                    }
                }
            }
#pragma unroll
            for (int d = 0; d < kDt; ++d) {
                const int n = i4 * kDt + d;
                if (n + kAheadV < 4 * kDt) read_v(n + kAheadV);
                __builtin_amdgcn_sched_barrier(kVMask);
#pragma unroll
                for (int u = kP - 1; u >= 0; --u)
                    o[d] = mfma32(vf[n % (kAheadV + 1)], p[u], o[d]);
            }
        }
        __builtin_amdgcn_s_setprio(0);
        if (more) finish(i + 1, buf ^ 1, next_edge);
        edge = next_edge;
        none = next_none;
        lds_barrier();
    }

    if (odd) {
        for (int i = 0; i < rows; ++i) {
            const int64_t rr = row0 + i;
            const int tk = (int)(rr / G), h = kvh * G + (int)(rr - (int64_t)tk * G);
            plain_row<INT8, FP32>(a, table, c0 + tk, h, kvh, len - (int)nq + tk, tile_token, i0, i1,
                            RowOut{(c0 + tk) * a.hq + h, part, parts}, reinterpret_cast<float *>(lds));
        }
        return;
    }

    l += __shfl_xor(l, 32, kWave);
    if (parts > 1) {
        if (!on) return;
        float *to = RowOut{(c0 + tok) * a.hq + head, part, parts}.sums(a);
#pragma unroll
        for (int d = 0; d < kDt; ++d)
#pragma unroll
            for (int r4 = 0; r4 < 4; ++r4) {
                const int at = d * 32 + 8 * r4 + 4 * half;
                if (at < D)
                    *reinterpret_cast<float4 *>(to + at) = float4{
                        o[d][4 * r4], o[d][4 * r4 + 1], o[d][4 * r4 + 2], o[d][4 * r4 + 3]};
            }
        if (half == 0) to[D] = INT8 ? m - kShift : m, to[D + 1] = l;
        return;
    }

    // O^T -> rows through LDS (the tiles are done), then whole rows to memory
    const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
    constexpr int kE = FP32 ? 4 : 2, kOut = DP * kE + 16;
    uint8_t *ob = lds + wave * 32 * kOut;
#pragma unroll
    for (int d = 0; d < kDt; ++d)
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
            const float4 y = {o[d][4 * r4] * inv, o[d][4 * r4 + 1] * inv, o[d][4 * r4 + 2] * inv,
                              o[d][4 * r4 + 3] * inv};
            uint8_t *to = ob + col * kOut + (d * 32 + 8 * r4 + 4 * half) * kE;
            if constexpr (FP32)
                *reinterpret_cast<float4 *>(to) = y;
            else
                *reinterpret_cast<uint2 *>(to) = uint2{pack_bf16(y.x, y.y), pack_bf16(y.z, y.w)};
        }
    __syncthreads();
    const int per_row = D * kE / 16;  // 16-byte pieces of a row
    for (int at = lane; at < 32 * per_row; at += kWave) {
        const int r = at / per_row, x = at - r * per_row;
        if (wave * 32 + r >= rows) break;
        const int64_t rr = row0 + wave * 32 + r;
        const int64_t tk = rr / G;
        const int64_t to = ((c0 + tk) * a.hq + kvh * G + (rr - tk * G)) * D * kE + x * 16;
        *reinterpret_cast<uint4 *>(reinterpret_cast<uint8_t *>(a.out) + to) =
            *reinterpret_cast<const uint4 *>(ob + r * kOut + x * 16);
    }
}

// Joins the parts of every row: D / 4 lanes have a row's values, 4 each, and 4
// groups of them take a quarter of the parts each, all loads at once (the time is
// one trip to memory: 3.9 us for 16 parts, 4.8 with four trips), joined in a fixed
// order through LDS.
template <bool FP32>
__global__ __launch_bounds__(256) void k_kv_prefill_join(KvAttnArgs a, int parts) {
    constexpr int kGroups = 4;
    __shared__ float4 so[256];
    __shared__ float sm[256], sl[256];
    const int tid = threadIdx.x;
    const int D = a.c.D, lanes = D / 4, rows = 256 / (kGroups * lanes);
    const int64_t row = (int64_t)blockIdx.x * rows + tid / (kGroups * lanes), all = a.T * a.hq;
    const int grp = tid / lanes % kGroups, d = tid % lanes * 4;
    constexpr int kEach = kMaxParts / kGroups;
    float mk[kEach], lk[kEach];
    float4 z[kEach];
#pragma unroll
    for (int x = 0; x < kEach; ++x) {
        const int i = grp + x * kGroups;
        const float *p = RowOut{min(row, all - 1), min(i, parts - 1), parts}.sums(a);
        mk[x] = p[D], lk[x] = p[D + 1];
        z[x] = *reinterpret_cast<const float4 *>(p + d);
    }
    // (while they are in flight) the row's sequence: nobody wrote the parts of a row
    // that belongs to none, and its output is left as it is
    const int64_t token = row / a.hq;
    const int64_t first = (int64_t)blockIdx.x * rows + tid / kWave * kWave / (kGroups * lanes);
    int64_t b = find_sequence(a.cu, a.B, min(first, all - 1) / a.hq);
    while (b + 1 < a.B && a.cu[b + 1] <= token) ++b;
    const int64_t c0 = a.cu[b], c1 = a.cu[b + 1];
    const bool on = tid < rows * kGroups * lanes && row < all && c0 >= 0 && c1 <= a.T &&
                    token >= c0 && token < c1;
    float m = -INFINITY, l = 0.0f;
    float4 y = {};
#pragma unroll
    for (int x = 0; x < kEach; ++x)
        if (grp + x * kGroups < parts) add_part(m, l, y, mk[x], lk[x], z[x]);
    so[tid] = y, sm[tid] = m, sl[tid] = l;
    __syncthreads();
    if (!on || grp) return;
#pragma unroll
    for (int g = 1; g < kGroups; ++g) {
        const int at = tid + g * lanes;
        add_part(m, l, y, sm[at], sl[at], so[at]);
    }
    store_out<FP32>(a.out, row * D + d, y, l);
}

namespace {

// Workgroups of a call for each part: tiles of 128 rows that its tokens can make.
int64_t row_tiles(int64_t T, int64_t B, int64_t G) { return T * G / kRows + B; }

// Few workgroups leave the chip idle and run through their tokens one tile after
// another: their tiles are then split over up to kMaxParts parts, as many as two
// workgroups a CU take, and joined by a second launch (3 chunks of up to 37 tokens
// behind up to 1001, fp32, 12 / 4 heads of 64: 36 us in one part, 13.5 us split).
// us of one chunk, 4 query heads a cache head of 128, bf16, in one part / up to 256 /
// 512 / 1024 workgroups:
//   rows, cache heads   behind 64                   1024                        16384 tokens
//      1, 2              8.7 / 10.0 / 10.0 / 10.0   26.5 / 11.5 / 11.5 / 11.5   309 / 29 / 29 / 29
//    128, 8             12.0 / 17.0 / 17.2 / 17.0   29.8 / 22.8 / 27.1 / 29.8   314 / 67 / 55 / 55
//    512, 8             19.8 / 19.4 / 37.1 / 41.4   37.2 / 37.1 / 42.8 / 48.3   322 / 322 / 172 / 171
// 512 is for the long contexts, where it saves most; many rows behind few tokens pay
// for it, since the host does not know the lengths.
constexpr int64_t kPartBlocks = 512;
int64_t most_parts(int64_t T, int64_t B, int64_t hq, int64_t heads) {
    const int64_t groups = row_tiles(T, B, hq / heads) * heads;
    return std::min<int64_t>(std::max<int64_t>(kPartBlocks / groups, 1), kMaxParts);
}

template <int DP, bool INT8, bool FP32>
hipError_t launch_dp(const KvAttnArgs &a, const char **path, hipStream_t st) {
    const int64_t groups = row_tiles(a.T, a.B, a.hq / a.c.heads) * a.c.heads;
    // tiles of the longest sequence that the table can hold and the window shows
    int64_t most = a.c.W << a.c.shift;
    if (a.window) most = std::min<int64_t>(most, (int64_t)a.window + a.sinks + kRows + 2 * kTile);
    const int parts = (int)std::min(most_parts(a.T, a.B, a.hq, a.c.heads), (most + kTile - 1) / kTile);
    const size_t tile_bytes = 2 * 2 * kTile * DP * 2;
    const size_t out_bytes = kRows * (DP * (FP32 ? 4 : 2) + 16);
    *path = parts > 1 ? "kv_prefill_split" : "kv_prefill";
    launch_kv(k_kv_prefill<DP, INT8, FP32>, dim3((unsigned)groups, parts), dim3(kThreads),
              std::max(tile_bytes, out_bytes), st, a, parts);
    if (parts > 1) {
        const int rows = 256 / a.c.D;  // of a workgroup: four groups of D / 4 lanes each
        hipLaunchKernelGGL(k_kv_prefill_join<FP32>,
                           dim3((unsigned)((a.T * a.hq + rows - 1) / rows)), dim3(256), 0, st, a,
                           parts);
    }
    return hipGetLastError();
}

template <int DP>
hipError_t launch_types(const KvAttnArgs &a, const char **path, hipStream_t st) {
    if (a.int8) return a.fp32 ? launch_dp<DP, true, true>(a, path, st) : launch_dp<DP, true, false>(a, path, st);
    return a.fp32 ? launch_dp<DP, false, true>(a, path, st) : launch_dp<DP, false, false>(a, path, st);
}

}  // namespace

// Bytes of the parts of every call of up to T tokens.  A larger call has fewer
// parts, so the most comes from the largest calls that still have p of them: those
// of one sequence whose workgroups are at most 512 / p.
size_t kv_prefill_ws_bytes(int64_t T, int64_t hq, int64_t heads, int64_t D) {
    int64_t rows = 0;
    for (int64_t p = 2; p <= kMaxParts; ++p) {
        const int64_t tiles = kPartBlocks / p / heads;  // T' * G / kRows + 1 at most
        if (tiles > 0)
            rows = std::max(rows, std::min(T, (tiles * kRows - 1) / (hq / heads)) * hq * p);
    }
    return (size_t)(rows * (D + 4) * 4);
}

hipError_t launch_kv_prefill(const KvAttnArgs &a, const char **path, hipStream_t st) {
    return a.c.D <= 64 ? launch_types<64>(a, path, st)
           : a.c.D <= 128 ? launch_types<128>(a, path, st)
                          : launch_types<256>(a, path, st);
}

}  // namespace w4
