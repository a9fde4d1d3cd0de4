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
// (the order of tokens inside its depth is free; V^T is laid out to match).
//
// K and V tiles go memory -> registers -> LDS, two LDS buffers, the loads of
// the next tile in flight during the products of this one, one barrier a tile.
// K lies row by row, V transposed (4 x VE blocks by byte permutes), both with
// 16-byte chunks XOR-swizzled so that reads of 16 rows cover all banks once.
// int8 codes become bf16 on the way to LDS (exact); their scales multiply the
// scores and the softmax weights.
#include "kv_attn.h"

namespace w4 {

namespace {

typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kRows = 128, kTile = 64, kThreads = 256;

__device__ __forceinline__ v16f mfma32(uint4 a, uint4 b, v16f c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a),
                                                   __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// Byte offset of 16-byte chunk `chunk` of token `t` in a K tile.
template <int DP>
__device__ __forceinline__ int k_at(int t, int chunk) {
    const int x = DP == 64 ? (t >> 1) & 7 : t & 15;
    return t * DP * 2 + ((chunk ^ x) << 4);
}

// Byte offset of chunk `chunk` (8 token places) of value d in a V^T tile.
// Place 8 h + j of the 16 tokens of chunks 2 i, 2 i + 1 is token
// 16 i + 8 (j / 4) + 4 h + j % 4: what lane half h holds of S^T.
__device__ __forceinline__ int v_at(int d, int chunk) {
    return d * kTile * 2 + ((chunk ^ ((d ^ (d >> 3) ^ (d >> 6)) & 7)) << 4);
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

// Loads of one K / V tile in registers.  Thread t has K chunks t % kCh of rows
// t / kCh + ..., and V values (t % 16) VE ... of the tokens 4 (t / 16) ... + 3.
template <int DP, bool INT8>
struct Stage {
    static constexpr int kB = INT8 ? 1 : 2;
    static constexpr int kCh = DP * kB / 16;           // 16-byte chunks of a row
    static constexpr int kLoads = kTile * kCh / kThreads;
    static constexpr int kStep = kThreads / kCh;       // rows between a thread's loads
    static constexpr int VE = DP / 16;
    static constexpr int kW = VE * kB / 4;             // dwords of a V piece
    u32x4 k[kLoads];
    uint32_t v[4][kW];
    float ks, vs;
    int bad;  // tokens (bits 0 .. 3) of v that no row of the workgroup sees
};

// One query row without the matrix cores, token by token, so that a token the
// row does not see takes no part at all: for workgroups whose edge tiles hold
// infinities or NaN in V (the products of a tile would carry them to every
// row as 0 * inf).  bf16 cache; the whole workgroup, `buf` 516 floats of LDS.
template <bool FP32>
__device__ void plain_row(const KvAttnArgs &a, const int32_t *table, int64_t token, int h, int kvh,
                          int pos, float *buf) {
    float *q = buf, *p = buf + 256, *red = buf + 512;
    const int tid = threadIdx.x, D = a.c.D;
    const int low = a.window ? pos - a.window + 1 : 0;
    __syncthreads();
    if (tid < D) {
        const int64_t at = token * a.ldq + (int64_t)h * D + tid;
        q[tid] = FP32 ? reinterpret_cast<const float *>(a.q)[at]
                      : bf16_lo(reinterpret_cast<const uint16_t *>(a.q)[at]);
    }
    const uint16_t *ck = reinterpret_cast<const uint16_t *>(a.c.k);
    const uint16_t *cv = reinterpret_cast<const uint16_t *>(a.c.v);
    auto vector = [&](int t) {
        const int pg = kv_page(a.c, table, t);
        return pg < 0 ? (int64_t)-1 : kv_vector(a.c, pg, kvh, t);
    };
    float m = -INFINITY, l = 0.0f, o = 0.0f;
    for (int t0 = 0; t0 <= pos; t0 += 256) {
        if (t0 + 256 <= low && t0 >= a.sinks) continue;
        __syncthreads();
        const int t = t0 + tid;
        const bool see = t <= pos && (t >= low || t < a.sinks);
        const int64_t vec = see ? vector(t) : -1;
        float s = -INFINITY;
        if (vec >= 0) {
            float x = 0.0f;
            for (int d = 0; d < D; ++d) x = __builtin_fmaf(q[d], bf16_lo(ck[vec * D + d]), x);
            s = x * a.scale;
        }
        const float mx = wave_max(s);
        if (tid % kWave == 0) red[tid / kWave] = mx;
        __syncthreads();
        const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
        const float alpha = mn == -INFINITY ? 1.0f : expf(m - mn);
        p[tid] = vec >= 0 ? expf(s - mn) : -1.0f;  // (-1: not seen)
        __syncthreads();
        m = mn;
        l *= alpha;
        o *= alpha;
        for (int j = 0; j < 256; ++j) {
            if (p[j] < 0.0f) continue;
            l += p[j];
            const int64_t vj = vector(t0 + j);
            if (tid < D) o = __builtin_fmaf(p[j], bf16_lo(cv[vj * D + tid]), o);
        }
    }
    if (tid < D) {
        const float y = l == 0.0f ? 0.0f : o / l;
        const int64_t at = (token * a.hq + h) * D + tid;
        if constexpr (FP32)
            reinterpret_cast<float *>(a.out)[at] = y;
        else
            reinterpret_cast<__bf16 *>(a.out)[at] = (__bf16)y;
    }
}

}  // namespace

template <int DP, bool INT8, bool FP32>
__global__ __launch_bounds__(kThreads, DP <= 128 && !FP32 ? 2 : 1) void k_kv_prefill(KvAttnArgs a) {
    using St = Stage<DP, INT8>;
    constexpr int kSteps = DP / 16, kDt = DP / 32, VE = St::VE;
    constexpr int kQ = FP32 ? 3 : 1, kP = kQ;
    constexpr int kKBytes = kTile * DP * 2, kBuf = 2 * kKBytes;
    extern __shared__ __align__(16) uint8_t lds[];
    __shared__ float sks[2][kTile], svs[2][kTile];
    __shared__ int odd;  // whether a tile at an edge has values of V that are not finite

    const int tid = threadIdx.x, lane = tid % kWave, half = lane / 32, col = lane % 32;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int D = a.c.D, G = a.hq / a.c.heads;
    const int kvh = (int)(blockIdx.x % a.c.heads);
    const int64_t idx = (int64_t)gridDim.x / a.c.heads - 1 - blockIdx.x / a.c.heads;
    const int64_t b = find_tile(a, G, idx);
    const int64_t c0 = a.cu[b];
    const int64_t nq = (int64_t)a.cu[b + 1] - c0;
    const int64_t row0 = (idx - first_tile(a, G, b)) * kRows;
    if (c0 < 0 || nq <= 0 || c0 + nq > a.T || row0 >= nq * G) return;

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
    const float scale2 = a.scale * 1.44269504088896340736f;

    // q stays in registers as the B operand, but for the three terms of 256 dims
    // (192 registers beside 128 of O): those are read and split for every tile
    constexpr bool kKeep = !(FP32 && DP == 256);
    const int64_t q_at = (c0 + tok) * a.ldq + head * D + half * 8;
    uint4 q[kQ][kKeep ? kSteps : 1];
    if constexpr (kKeep)
#pragma unroll
        for (int j = 0; j < kSteps; ++j)
            load_query<FP32>(a.q, q_at + j * 16, on && j * 16 + half * 8 < D, q, j);

    auto tile_token = [&](int i) {
        return kTile * (i < sink_tiles ? i : i - sink_tiles + lo_tile);
    };
    // pages of the four 16-token quarters of a tile (-1: none)
    auto tile_pages = [&](int t0, int (&page)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) page[j] = kv_page(a.c, table, t0 + 16 * j);
    };
    // whether some row does not see some token of the tile
    auto at_edge = [&](int t0, const int (&page)[4]) {
        return t0 + kTile - 1 > pos0 || (a.window && t0 < low1 && t0 + kTile > a.sinks) ||
               (page[0] | page[1] | page[2] | page[3]) < 0;
    };
    auto load = [&](St &st, int t0, const int (&page)[4]) {
#pragma unroll
        for (int j = 0; j < St::kLoads; ++j) {
            const int t = tid / St::kCh + j * St::kStep, ch = tid % St::kCh;
            // (a wave's rows of one load lie in one quarter)
            const int qt = __builtin_amdgcn_readfirstlane(t / 16);
            const int pg = qt == 0 ? page[0] : qt == 1 ? page[1] : qt == 2 ? page[2] : page[3];
            const int64_t vec = kv_vector(a.c, max(pg, 0), kvh, t0 + 16 * qt) + t % 16;
            const int d = ch * (16 / St::kB);
            st.k[j] = *reinterpret_cast<const u32x4 *>(a.c.k + (vec * D + (d < D ? d : 0)) * St::kB);
        }
        const int pg = wave == 0 ? page[0] : wave == 1 ? page[1] : wave == 2 ? page[2] : page[3];
        const int64_t vec0 = kv_vector(a.c, max(pg, 0), kvh, t0 + 16 * wave);
        const int t = lane / 16 * 4, d = lane % 16 * VE;
        const uint8_t *vp = a.c.v + ((vec0 + t) * D + (d < D ? d : 0)) * St::kB;
        st.bad = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int w = 0; w < St::kW; w += St::kW < 4 ? St::kW : 4) {
                const uint8_t *p = vp + j * D * St::kB + w * 4;
                if constexpr (St::kW >= 4) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(p);
                    st.v[j][w] = x.x, st.v[j][w + 1] = x.y;
                    st.v[j][w + 2] = x.z, st.v[j][w + 3] = x.w;
                } else if constexpr (St::kW == 2) {
                    const uint2 x = *reinterpret_cast<const uint2 *>(p);
                    st.v[j][0] = x.x, st.v[j][1] = x.y;
                } else {
                    st.v[j][0] = *reinterpret_cast<const uint32_t *>(p);
                }
            }
            const int tj = t0 + 16 * wave + t + j;
            const bool seen = tj <= pos1 && (tj >= low0 || tj < a.sinks) && pg >= 0;
            if (!seen) st.bad |= 1 << j;
        }
        if constexpr (INT8) {
            // lanes 0 .. 15 of a wave: the scales of its 16 tokens
            st.ks = a.c.ks[vec0 + lane % 16];
            st.vs = a.c.vs[vec0 + lane % 16];
        }
    };
    auto store = [&](St &st, int buf, bool edge) {
        uint8_t *kb = lds + buf * kBuf, *vb = kb + kKBytes;
#pragma unroll
        for (int j = 0; j < St::kLoads; ++j) {
            const int t = tid / St::kCh + j * St::kStep, ch = tid % St::kCh;
            if constexpr (INT8) {
                *reinterpret_cast<uint4 *>(kb + k_at<DP>(t, 2 * ch)) = codes8(__builtin_bit_cast(uint4, st.k[j]), 0);
                *reinterpret_cast<uint4 *>(kb + k_at<DP>(t, 2 * ch + 1)) = codes8(__builtin_bit_cast(uint4, st.k[j]), 1);
            } else {
                *reinterpret_cast<u32x4 *>(kb + k_at<DP>(t, ch)) = st.k[j];
            }
        }
        if (edge) {
            // values that no row sees may be anything: clear them; those that
            // some rows see and others do not must be finite for the product
            // with a weight of zero: note where they are not
            bool inf = false;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int w = 0; w < St::kW; ++w) {
                    if (st.bad >> j & 1) st.v[j][w] = 0;
                    if constexpr (!INT8)
                        inf |= (st.v[j][w] & 0x7F80u) == 0x7F80u ||
                               (st.v[j][w] & 0x7F800000u) == 0x7F800000u;
                }
            if (inf) odd = 1;
        }
        const int t4 = lane / 16;  // tokens 4 t4 .. + 3 of the wave's 16
        const int chunk = wave * 2 + t4 % 2, sub = t4 / 2 * 8;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            uint2 x;
            if constexpr (INT8) {
                const int w = e / 4, s = e % 4 * 8;
                x.x = code_pair((int8_t)(st.v[0][w] >> s), (int8_t)(st.v[1][w] >> s));
                x.y = code_pair((int8_t)(st.v[2][w] >> s), (int8_t)(st.v[3][w] >> s));
            } else {
                const uint32_t sel = e % 2 ? 0x07060302u : 0x05040100u;
                x.x = __builtin_amdgcn_perm(st.v[1][e / 2], st.v[0][e / 2], sel);
                x.y = __builtin_amdgcn_perm(st.v[3][e / 2], st.v[2][e / 2], sel);
            }
            *reinterpret_cast<uint2 *>(vb + v_at(lane % 16 * VE + e, chunk) + sub) = x;
        }
        if constexpr (INT8) {
            if (lane < 16) {
                sks[buf][wave * 16 + lane] = st.ks;
                svs[buf][wave * 16 + lane] = st.vs;
            }
        }
    };

    if (tid == 0) odd = 0;
    __syncthreads();
    v16f o[kDt] = {};
    float m = -INFINITY, l = 0.0f;
    St st;
    int page[4], next[4] = {};
    bool edge = false;
    if (tiles > 0) {
        const int t0 = tile_token(0);
        tile_pages(t0, page);
        edge = at_edge(t0, page);
        load(st, t0, page);
        store(st, 0, edge);
    }
    __syncthreads();
    for (int i = 0; i < tiles; ++i) {
        const int buf = i & 1;
        const int t0 = tile_token(i);
        bool next_edge = false;
        if (i + 1 < tiles) {
            const int t1 = tile_token(i + 1);
            tile_pages(t1, next);
            next_edge = at_edge(t1, next);
            load(st, t1, next);
        }
        const uint8_t *kb = lds + buf * kBuf, *vb = kb + kKBytes;
        v16f s[2] = {};
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            if constexpr (!kKeep)
                load_query<FP32>(a.q, q_at + j * 16, on && j * 16 + half * 8 < D, q, 0);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint4 kk = *reinterpret_cast<const uint4 *>(
                    kb + k_at<DP>(t * 32 + col, j * 2 + half));
#pragma unroll
                for (int u = kQ - 1; u >= 0; --u) s[t] = mfma32(kk, q[u][kKeep ? j : 0], s[t]);
            }
        }
        // scores in units of log 2; token of register r: 32 t + 8 (r / 4) + 4 half + r % 4
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r4 = 0; r4 < 4; ++r4) {
                float4 ks = {1.0f, 1.0f, 1.0f, 1.0f};
                if constexpr (INT8)
                    ks = *reinterpret_cast<const float4 *>(&sks[buf][32 * t + 8 * r4 + 4 * half]);
                s[t][4 * r4] *= INT8 ? scale2 * ks.x : scale2;
                s[t][4 * r4 + 1] *= INT8 ? scale2 * ks.y : scale2;
                s[t][4 * r4 + 2] *= INT8 ? scale2 * ks.z : scale2;
                s[t][4 * r4 + 3] *= INT8 ? scale2 * ks.w : scale2;
            }
        if (edge) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int tj = t0 + 32 * t + 8 * (r / 4) + 4 * half + r % 4;
                    const bool see = tj <= pos && (tj >= low || tj < a.sinks) &&
                                     page[2 * t + r / 8] >= 0;
                    if (!see) s[t][r] = -INFINITY;
                }
        }
        float mt = s[0][0];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) mt = fmaxf(mt, s[t][r]);
        mt = fmaxf(mt, __shfl_xor(mt, 32, kWave));
        if (__any(mt > m)) {
            const float mn = fmaxf(m, mt);
            const float alpha = m == mn ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= alpha;
#pragma unroll
            for (int d = 0; d < kDt; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[d][r] *= alpha;
        }
        const float mu = m == -INFINITY ? 0.0f : m;
        uint4 p[kP][4];
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) {  // 16 tokens: registers 8 (i4 % 2) ... of half i4 / 2
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float e = __builtin_amdgcn_exp2f(s[i4 / 2][8 * (i4 % 2) + j] - mu);
                l += e;
                f[j] = e;
            }
            if constexpr (INT8) {
#pragma unroll
                for (int j4 = 0; j4 < 2; ++j4) {
                    const float4 v = *reinterpret_cast<const float4 *>(
                        &svs[buf][16 * i4 + 8 * j4 + 4 * half]);
                    // (a weight of zero stays zero whatever an unseen token's scale is)
                    f[4 * j4] = f[4 * j4] == 0.0f ? 0.0f : f[4 * j4] * v.x;
                    f[4 * j4 + 1] = f[4 * j4 + 1] == 0.0f ? 0.0f : f[4 * j4 + 1] * v.y;
                    f[4 * j4 + 2] = f[4 * j4 + 2] == 0.0f ? 0.0f : f[4 * j4 + 2] * v.z;
                    f[4 * j4 + 3] = f[4 * j4 + 3] == 0.0f ? 0.0f : f[4 * j4 + 3] * v.w;
                }
            }
            uint4 w[kP];
            split_bf16<kP>(f, w);
#pragma unroll
            for (int u = 0; u < kP; ++u) p[u][i4] = w[u];
        }
#pragma unroll
        for (int d = 0; d < kDt; ++d)
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4) {
                const uint4 vv = *reinterpret_cast<const uint4 *>(
                    vb + v_at(d * 32 + col, i4 * 2 + half));
#pragma unroll
                for (int u = kP - 1; u >= 0; --u) o[d] = mfma32(vv, p[u][i4], o[d]);
            }
        if (i + 1 < tiles) store(st, buf ^ 1, next_edge);
        edge = next_edge;
#pragma unroll
        for (int j = 0; j < 4; ++j) page[j] = next[j];
        __syncthreads();
    }

    if (!INT8 && odd) {
        for (int i = 0; i < rows; ++i) {
            const int64_t rr = row0 + i;
            const int tk = (int)(rr / G), h = kvh * G + (int)(rr - (int64_t)tk * G);
            plain_row<FP32>(a, table, c0 + tk, h, kvh, len - (int)nq + tk,
                            reinterpret_cast<float *>(lds));
        }
        return;
    }

    // O^T -> rows through LDS (the tiles are done), then whole rows to memory
    l += __shfl_xor(l, 32, kWave);
    const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
    constexpr int kE = FP32 ? 4 : 2, kPitch = DP * kE + 16;
    uint8_t *ob = lds + wave * 32 * kPitch;
#pragma unroll
    for (int d = 0; d < kDt; ++d)
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
            const float4 y = {o[d][4 * r4] * inv, o[d][4 * r4 + 1] * inv, o[d][4 * r4 + 2] * inv,
                              o[d][4 * r4 + 3] * inv};
            uint8_t *to = ob + col * kPitch + (d * 32 + 8 * r4 + 4 * half) * kE;
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
            *reinterpret_cast<const uint4 *>(ob + r * kPitch + x * 16);
    }
}

namespace {

template <int DP, bool INT8, bool FP32>
hipError_t launch_dp(const KvAttnArgs &a, hipStream_t st) {
    const int G = a.hq / a.c.heads;
    const int64_t tiles = a.T * G / kRows + a.B;
    const size_t tile_bytes = 2 * 2 * kTile * DP * 2;
    const size_t out_bytes = kRows * (DP * (FP32 ? 4 : 2) + 16);
    hipLaunchKernelGGL((k_kv_prefill<DP, INT8, FP32>), dim3((unsigned)(tiles * a.c.heads)),
                       dim3(kThreads), std::max(tile_bytes, out_bytes), st, a);
    return hipGetLastError();
}

template <int DP>
hipError_t launch_types(const KvAttnArgs &a, hipStream_t st) {
    if (a.int8) return a.fp32 ? launch_dp<DP, true, true>(a, st) : launch_dp<DP, true, false>(a, st);
    return a.fp32 ? launch_dp<DP, false, true>(a, st) : launch_dp<DP, false, false>(a, st);
}

}  // namespace

hipError_t launch_kv_prefill(const KvAttnArgs &a, hipStream_t st) {
    return a.c.D <= 64 ? launch_types<64>(a, st)
           : a.c.D <= 128 ? launch_types<128>(a, st)
                          : launch_types<256>(a, st);
}

}  // namespace w4
