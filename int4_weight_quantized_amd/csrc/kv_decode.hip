// Attention of one new token per sequence over the paged key-value cache.
//
//   s_j = scale <q, k_j>,  o = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
//
// One pass over K and V with a running maximum m and sum.  Bound by memory:
// every visible token's K and V are read once and meet G = q_heads / heads
// query rows, 2 G flops a byte, so the matrix cores have time to spare.
//
// The rows are padded to the 16 columns of v_mfma_f32_16x16x32_bf16, and both
// products are taken transposed, S^T = K Q^T and O^T = V^T P^T: the
// accumulators of S^T (lane = query row, registers = tokens) are then the
// B operand of the second product as they stand.  The order of the tokens
// inside that product's depth of 32 is free, so lane group g takes tokens
// 4g .. 4g+3 of both 16-token halves and P never leaves its lane.  Softmax
// maxima and rescaling are one value a lane.
//
// K and V are read in whole rows with non-temporal loads (each byte is used
// once; half rows, as the A operand wants K, made every line two requests).  K
// goes through 16 rows of the wave's own LDS into the A operand, V is transposed
// by byte permutes of register pairs.  No barrier in the loop: the waves of a
// workgroup take tiles of 32 tokens in turn and are joined through LDS once per
// (sequence, cache head).
//
// fp32 activations: q and the softmax weights are split into three bf16 terms
// (24 significant bits), each its own MFMA into the same fp32 accumulator; K
// and V are exact in bf16 (int8 codes have 8 bits), so products keep fp32
// accuracy.  bf16 activations: q is exact, the weights keep two terms (16
// bits), so that the output's own rounding dominates.  Where the group's rows
// leave columns free (4 rows of 3 terms, 8 rows of 2), the terms take columns
// of their own: one MFMA for all of them, and the columns are summed at the end.
//
// Bound by memory.  4 sequences of 131072 tokens, 64 / 8 heads of 128, bf16: 330
// us, 6.5 TB/s (a plain read: 7.05; this kernel's loads without its products: 325
// us).  64 ragged sequences up to 8191, 32 / 8 heads, int8, fp32 activations: 99
// us, 5.3 TB/s (a tile of int8 has half the bytes of one of bf16 in flight, and the
// same work).  One token behind 700 with a window of 512, 4 / 1 heads of 256: 10.5
// us, one workgroup's three rounds of tiles one after another.
#include "kv_attn.h"

namespace w4 {

namespace {

constexpr int kRowRor4 = 0x124;  // row_ror:4

__device__ __forceinline__ v4f mfma16(uint4 a, uint4 b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                   __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// The tokens that a position sees, as tiles of 32: the first `sink_tiles`
// tiles, then the tiles from lo / 32 to the end.
struct Span {
    int n, lo;  // tokens 0 <= j < n with j >= lo or j < sinks
    int sink_tiles, lo_tile, tiles;
};

__device__ __forceinline__ Span make_span(const KvAttnArgs &a, int64_t b) {
    Span s;
    s.n = kv_length(a, b);
    s.lo = a.window ? max(s.n - a.window, 0) : 0;
    s.lo_tile = s.lo / 32;
    s.sink_tiles = min((a.sinks + 31) / 32, s.lo_tile);
    s.tiles = s.sink_tiles + (s.n + 31) / 32 - s.lo_tile;
    return s;
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// One lane's VD consecutive values of a row.
template <bool INT8, int VD>
struct Piece {
    static constexpr int kWords = VD * (INT8 ? 1 : 2) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const uint8_t *p) {
        if constexpr (kWords == 1) {
            w[0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t *>(p));
        } else if constexpr (kWords == 2) {
            const u32x2 x = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(p));
            w[0] = x[0], w[1] = x[1];
        } else {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const u32x4 x =
                    __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p + 4 * i));
                w[i] = x[0], w[i + 1] = x[1], w[i + 2] = x[2], w[i + 3] = x[3];
            }
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
};

// Value e of two pieces as a bf16 pair.
template <bool INT8, int VD>
__device__ __forceinline__ uint32_t pair(const Piece<INT8, VD> &x, const Piece<INT8, VD> &y,
                                         int e) {
    if constexpr (INT8)
        return code_pair((int8_t)(x.w[e / 4] >> (e % 4 * 8)), (int8_t)(y.w[e / 4] >> (e % 4 * 8)));
    else
        return __builtin_amdgcn_perm(y.w[e / 2], x.w[e / 2], e % 2 ? 0x07060302u : 0x05040100u);
}

// Sum over the 16 / N groups of N columns (N = 4, 8); every lane gets it, with
// the same bits in every group.
template <int N>
__device__ __forceinline__ float sum_columns(float v) {
    v += __int_as_float(dpp<kRowRor8>(__float_as_int(v)));
    if constexpr (N == 4) v += __int_as_float(dpp<kRowRor4>(__float_as_int(v)));
    return v;
}

// Term `term` of the split_bf16 of eight floats (zeros from N on): every lane
// its own, by leaving out the subtractions behind it.
template <int N>
__device__ __forceinline__ uint4 term_bf16(const float (&f)[8], int term) {
    float r[8];
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = f[j];
#pragma unroll
    for (int t = 0; t < N; ++t) {
        const float on = t < term ? -1.0f : 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = pack_bf16(r[2 * j], r[2 * j + 1]);
            if (t + 1 < N) {
                r[2 * j] = __builtin_fmaf(on, bf16_lo(w[j]), r[2 * j]);
                r[2 * j + 1] = __builtin_fmaf(on, bf16_hi(w[j]), r[2 * j + 1]);
            }
        }
    }
    const bool none = term >= N;
    return uint4{none ? 0 : w[0], none ? 0 : w[1], none ? 0 : w[2], none ? 0 : w[3]};
}

// A wave's 32 tokens.
template <int DP, bool INT8>
struct Tile {
    u32x4 k[2][INT8 ? DP / 64 : DP / 32];
    Piece<INT8, DP / 16> v[2][4];
    v4f ks[2], vs[2];
};

__device__ __forceinline__ int clamp_dim(int d, int D) { return d < D ? d : 0; }

// Where they are: the first token, the pages of its halves and their first vectors.
struct Place {
    int t0, page[2];
    int64_t vec[2];
};

// Byte offset of 16-byte chunk `ch` of row `row` among 16 rows of kCh chunks,
// XOR-swizzled so that 16 rows' chunks of one index cover all banks once.
template <int kCh>
__device__ __forceinline__ int stage_at(int row, int ch) {
    return row * kCh * 16 + ((ch ^ (kCh == 8 ? row >> 1 & 7 : row & 15)) << 4);
}

// The split kernel: workgroups of 4 waves, 3 a CU of the 256 in one round (512
// workgroups: 136 us where 768 take 122 and 1536 136; 64 ragged sequences, int8).
constexpr int kSplitWaves = 4, kSplitBlocks = 768;

// Waves a SIMD that the registers are cut to: as many as K, V, q and O of a
// wave leave room for without spilling much.
constexpr int waves_per_simd(int DP, bool INT8, bool FP32, bool PACK) {
    return DP == 256 ? (FP32 && !PACK ? 1 : 2) : DP == 128 ? (FP32 && !PACK && !INT8 ? 2 : 3) : 4;
}

template <int NW>
__device__ __forceinline__ int pair_units(const Span &s) {
    return max((s.tiles + NW - 1) / NW, 1);
}

// Query heads in groups of up to 16 that share a cache head: `per_head` groups
// for each of the cache's heads, `rows` rows at most in one.  Each group reads K and
// V for itself (4 sequences of 131072 tokens, 8 cache heads of 128, bf16: 330 us for
// 64 query heads, 339 for 128, 656 for 256).
struct KvHeads {
    int group, rows, per_head, count;
    __host__ __device__ explicit KvHeads(const KvAttnArgs &a) {
        group = a.hq / a.c.heads;
        rows = group < 16 ? group : 16;
        per_head = (group + 15) / 16;
        count = per_head * a.c.heads;
    }
};

// Work of the split kernel.  A unit is one tile for each of NW waves of one
// (sequence, head) pair; a pair costs its units and kStart more (its start and
// its join keep a workgroup about as long; 0, 1, 2, 3, 4: 122, 113, 105, 106, 110
// us on 64 ragged sequences).  Pairs follow one
// another, sequence-major, and the cost U of all of them is dealt to the first
// n = min(workgroups, U) workgroups in equal runs: workgroup k has the places
// floor(k U / n) to floor((k + 1) U / n), whatever the lengths are; the first
// kStart places of a pair hold no unit.  A sequence without tokens has one
// unit (its outputs are zeros).
constexpr int kStart = 2;

struct KvCursor {
    int64_t b;     // the pair
    int h, at;     // the head, the first place of the pair
    int left;      // places left of the run
};

__device__ __forceinline__ int64_t uniform(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(v >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// Cost of a pair of sequence b0 + lane, and the running sum over the lanes.
template <int NW>
__device__ __forceinline__ int64_t scan_cost(const KvAttnArgs &a, int64_t b0, int &cost) {
    const int lane = threadIdx.x % kWave;
    cost = b0 + lane < a.B ? pair_units<NW>(make_span(a, b0 + lane)) + kStart : 0;
    int64_t s = cost;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const int64_t t = __shfl_up(s, o, kWave);
        if (lane >= o) s += t;
    }
    return s;
}

template <int NW>
__device__ __forceinline__ KvCursor kv_first_segment(const KvAttnArgs &a, const KvHeads &hd,
                                                     int64_t k, int64_t n) {
    int64_t s = 0, U = 0, before = 0;
    int cost = 0;
    for (int64_t b0 = 0; b0 < a.B; b0 += kWave) {
        s = scan_cost<NW>(a, b0, cost);
        U += uniform(__shfl(s, kWave - 1, kWave));
    }
    U *= hd.count;
    n = min(n, U);
    if (k >= n) return KvCursor{0, 0, 0, 0};
    const int64_t first = k * U / n, last = (k + 1) * U / n;
    KvCursor cur{0, 0, 0, (int)(last - first)};
    for (int64_t b0 = 0; b0 < a.B; b0 += kWave) {
        if (a.B > kWave) s = scan_cost<NW>(a, b0, cost);
        // the first sequence whose places end behind `first`
        const uint64_t hit = __ballot((before + s) * hd.count > first);
        if (hit) {
            const int at = __ffsll((unsigned long long)hit) - 1;
            const int c = __builtin_amdgcn_readlane(cost, at);
            const int64_t off = first - (before + uniform(__shfl(s, at, kWave)) - c) * hd.count;
            cur.b = b0 + at;
            cur.h = (int)(off / c);
            cur.at = (int)(off - (int64_t)cur.h * c);
            return cur;
        }
        before += uniform(__shfl(s, kWave - 1, kWave));
    }
    cur.left = 0;  // (not reached: first < U)
    return cur;
}

// The part of a pair that a workgroup leaves in the workspace: unnormalized
// sums, maxima and sums of weights.  Slot 2 k + 1: workgroup k's part that
// starts a pair, slot 2 k: one that does not.
struct KvPartial {
    float *o, *m, *l;
    __device__ KvPartial(const KvAttnArgs &a, const KvHeads &hd, int DP, int64_t slot) {
        o = reinterpret_cast<float *>(static_cast<uint8_t *>(a.ws) + kSplitBlocks * 16) +
            slot * hd.rows * (DP + 4);
        m = o + hd.rows * DP;
        l = m + hd.rows;
    }
};

// At the workspace's start, for each workgroup: whether it has the first units of
// a pair, but not its last ones (then the pair), and whether its run begins with
// the last units of a pair that it did not start.  The workgroups between these
// two have nothing but units of that pair.
constexpr int kStarts = 1, kEnds = 2;
struct KvSplitPair {
    int64_t b;
    int h, flags;
};

}  // namespace

// DP: head_dim rounded up to 64, 128 or 256 (values beyond head_dim: q is zero
// there, and their V rows are not stored).  PACK: few rows (4 with fp32
// activations, 8 with bf16), whose terms share the 16 columns.  NW: waves.  SPLIT: the workgroups
// share all units of work evenly (see KvCursor), else workgroup i has all of
// (sequence, head) i.
template <int DP, bool INT8, bool FP32, bool PACK, int NW, bool SPLIT>
__global__ __launch_bounds__(
    NW * 64, waves_per_simd(DP, INT8, FP32, PACK)) void k_kv_decode(KvAttnArgs a) {
    constexpr int kSteps = DP / 32, VD = DP / 16, kB = INT8 ? 1 : 2;
    constexpr int kLoads = INT8 ? kSteps / 2 : kSteps;
    constexpr int kCh = DP * kB / 16, kRowsPer = 64 / kCh;  // 16-byte chunks of a row, rows of a load
    constexpr int kTerms = FP32 ? 3 : 2;                     // of the softmax weights
    constexpr int kQ = FP32 && !PACK ? 3 : 1, kP = PACK ? 1 : kTerms;
    constexpr int kGroup = PACK ? (FP32 ? 4 : 8) : 16;      // columns of one term
    constexpr int kRow = DP + 4;  // LDS row of the join, padded off the banks
    extern __shared__ float lds[];
    const int lane = threadIdx.x % kWave, c = lane % 16, g = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const KvHeads hd(a);
    // LDS: maxima and sums of the join, then its rows, in the same place as the
    // waves' K tiles of the loop (a barrier lies between)
    float *sm = lds, *sl = sm + NW * 16;
    float *join = sl + NW * 16;
    uint8_t *stage = reinterpret_cast<uint8_t *>(join) + wave * 16 * DP * kB;
    const float scale2 = a.scale * 1.44269504088896340736f;
    const int D = a.c.D;

    KvCursor cur = SPLIT ? kv_first_segment<NW>(a, hd, blockIdx.x, gridDim.x)
                         : KvCursor{(int64_t)blockIdx.x / hd.count, (int)(blockIdx.x % hd.count),
                                    0, 0x7FFFFFFF};
    KvSplitPair mark{0, 0, 0};
    while (cur.left > 0) {
        const int64_t b = cur.b;
        const Span sp = make_span(a, b);
        const int units = pair_units<NW>(sp);
        const int end = min(units + kStart - cur.at, cur.left) + cur.at;
        const int u0 = max(cur.at - kStart, 0), u1 = max(end - kStart, 0);
        if (u0 == u1) break;  // (the run ends in front of the pair's first unit)
        const int kvh = cur.h / hd.per_head, part = cur.h % hd.per_head;
        const int rows = min(hd.group - part * 16, 16);
        const int64_t qrow = b * a.ldq + ((int64_t)kvh * hd.group + part * 16) * D;

        // q as the B operand: lane c holds row c, group g its share of each 32 dims;
        // packed, lane c holds term c / kGroup of row c % kGroup
        const int term = c / kGroup, qr = c % kGroup;
        uint4 q[kQ][kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int d = INT8 ? s / 2 * 64 + g * 16 + s % 2 * 8 : s * 32 + g * 8;
            if constexpr (FP32 && PACK) {
                uint4 all[3][1];
                load_query<FP32>(a.q, qrow + (int64_t)qr * D + d, qr < rows && d < D, all, 0);
                auto pick = [&](uint32_t t0, uint32_t t1, uint32_t t2) {
                    return term == 0 ? t0 : term == 1 ? t1 : term == 2 ? t2 : 0u;
                };
                q[0][s].x = pick(all[0][0].x, all[1][0].x, all[2][0].x);
                q[0][s].y = pick(all[0][0].y, all[1][0].y, all[2][0].y);
                q[0][s].z = pick(all[0][0].z, all[1][0].z, all[2][0].z);
                q[0][s].w = pick(all[0][0].w, all[1][0].w, all[2][0].w);
            } else {
                load_query<FP32>(a.q, qrow + (int64_t)qr * D + d, qr < rows && d < D, q, s);
            }
        }
        v4f o[VD] = {};
        float m = -INFINITY, l = 0.0f;
        // int8: weights are 2^shift times as large where the wave's first scales of V
        // that are not zero are tiny, so that the terms of their products stay normal
        // numbers
        float shift = 0.0f;
        bool fresh = true;
        const int32_t *table = a.c.table + b * a.c.W;
        const int last = min(u1 * NW, sp.tiles);
        auto tile_token = [&](int i) {
            return 32 * (i < sp.sink_tiles ? i : i - sp.sink_tiles + sp.lo_tile);
        };
        // pages of this wave's next 32 tiles, one lane for each 16 tokens: one
        // load for all of them, off the path of the loads that need them
        int base = 0, pages = -1;
        auto look_up = [&](int i) {
            const int ii = i + lane / 2 * NW;
            base = i;
            pages = ii < last ? kv_page(a.c, table, tile_token(ii) + lane % 2 * 16) : -1;
        };
        Place now;
        auto place = [&](Place &p, int i) {
            if (i - base >= 32 * NW) look_up(i);
            const int at = (i - base) / NW * 2;
            p.t0 = tile_token(i);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                p.page[h] = __builtin_amdgcn_readlane(pages, at + h);
                p.vec[h] = kv_vector(a.c, max(p.page[h], 0), kvh, p.t0 + 16 * h);
            }
        };
        Tile<DP, INT8> t;
        // (a uniform address and a lane's 32-bit offset in a page: whole rows one
        // after another; rows of 64 bytes: one load has all 16, each lane its own
        // place of the A operand)
        const uint32_t k_off = ((kCh > 4 ? lane / kCh : c) * D + clamp_dim(
                                    (kCh > 4 ? lane % kCh : g) * (16 / kB), D)) * kB;
        const uint32_t v_off = (g * 4 * D + clamp_dim(c * VD, D)) * kB;
        auto load_k = [&](const Place &p, int h) {
            const uint8_t *at = a.c.k + p.vec[h] * (D * kB);
#pragma unroll
            for (int s = 0; s < kLoads; ++s, at += kRowsPer * D * kB)
                t.k[h][s] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(at + k_off));
        };
        auto load_ks = [&](const Place &p, int h) {
            if constexpr (INT8)
                t.ks[h] = *reinterpret_cast<const v4f *>(a.c.ks + p.vec[h] + (uint32_t)(g * 4));
        };
        auto load_v = [&](const Place &p) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t *at = a.c.v + p.vec[h] * (D * kB);
                if constexpr (INT8)
                    t.vs[h] = *reinterpret_cast<const v4f *>(a.c.vs + p.vec[h] + (uint32_t)(g * 4));
#pragma unroll
                for (int j = 0; j < 4; ++j, at += D * kB) t.v[h][j].load(at + v_off);
            }
        };
        auto compute = [&]() {
            float x[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // rows -> the A operand (lane: row c, chunk 4 s + g) through this
                // wave's LDS; a wave's LDS operations are in order
                u32x4 ka[kLoads];
                if constexpr (kCh > 4) {
#pragma unroll
                    for (int s = 0; s < kLoads; ++s)
                        *reinterpret_cast<u32x4 *>(
                            stage + stage_at<kCh>(s * kRowsPer + lane / kCh, lane % kCh)) = t.k[h][s];
                    __builtin_amdgcn_wave_barrier();
#pragma unroll
                    for (int s = 0; s < kLoads; ++s)
                        ka[s] = *reinterpret_cast<const u32x4 *>(stage + stage_at<kCh>(c, 4 * s + g));
                    __builtin_amdgcn_wave_barrier();
                } else {
                    ka[0] = t.k[h][0];
                }
                v4f s4 = {};
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    const uint4 raw = __builtin_bit_cast(uint4, ka[INT8 ? s / 2 : s]);
                    const uint4 kk = INT8 ? codes8(raw, s % 2) : raw;
#pragma unroll
                    for (int u = kQ - 1; u >= 0; --u) s4 = mfma16(kk, q[u][s], s4);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if constexpr (FP32 && PACK) s4[r] = sum_columns<kGroup>(s4[r]);
                    x[h][r] = s4[r] * (INT8 ? scale2 * t.ks[h][r] : scale2);
                }
            }
            // tiles at an edge, or with a page missing: hide tokens, and clear
            // their V, which may hold anything (0 * NaN would stay)
            if (now.t0 + 32 > sp.n || (now.t0 < sp.lo && now.t0 + 32 > a.sinks) ||
                (now.page[0] | now.page[1]) < 0) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int j = now.t0 + 16 * h + 4 * g + r;
                        const bool see =
                            j < sp.n && (j >= sp.lo || j < a.sinks) && now.page[h] >= 0;
                        if (!see) {
                            x[h][r] = -INFINITY;
                            t.v[h][r].zero();
                            if constexpr (INT8) t.vs[h][r] = 0.0f;
                        }
                    }
            }
            if (INT8 && fresh) {
                float big = 0.0f;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r) big = fmaxf(big, fabsf(t.vs[h][r]));
                big = fmaxf(big, __shfl_xor(big, 16, kWave));
                big = fmaxf(big, __shfl_xor(big, 32, kWave));
                if (__builtin_amdgcn_readfirstlane(big > 0.0f)) {
                    fresh = false;
                    if (__builtin_amdgcn_readfirstlane(big < 0x1p-60f)) shift = 40.0f, l *= 0x1p40f;
                }
            }
            float mt = x[0][0];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < 4; ++r) mt = fmaxf(mt, x[h][r]);
            mt = fmaxf(mt, __shfl_xor(mt, 16, kWave));
            mt = fmaxf(mt, __shfl_xor(mt, 32, kWave));
            if (__any(mt > m)) {
                const float mn = fmaxf(m, mt);
                const float alpha = m == mn ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
                m = mn;
                l *= alpha;
#pragma unroll
                for (int e = 0; e < VD; ++e)
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[e][r] *= alpha;
            }
            const float mu = m == -INFINITY ? 0.0f : m - shift;
            float p[8];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float e = __builtin_amdgcn_exp2f(x[h][r] - mu);
                    l += e;
                    p[4 * h + r] = INT8 ? e * t.vs[h][r] : e;
                }
            uint4 pb[kP];
            if constexpr (PACK)
                pb[0] = term_bf16<kTerms>(p, term);
            else
                split_bf16<kP>(p, pb);
#pragma unroll
            for (int e = 0; e < VD; ++e) {
                const uint4 vt = {pair(t.v[0][0], t.v[0][1], e), pair(t.v[0][2], t.v[0][3], e),
                                  pair(t.v[1][0], t.v[1][1], e), pair(t.v[1][2], t.v[1][3], e)};
#pragma unroll
                for (int u = kP - 1; u >= 0; --u) o[e] = mfma16(vt, pb[u], o[e]);
            }
        };
        int i = u0 * NW + wave;
        if (i < last) {
            look_up(i);
            for (; i < last; i += NW) {
                place(now, i);
#pragma unroll
                for (int h = 0; h < 2; ++h) load_k(now, h), load_ks(now, h);
                load_v(now);
                compute();
            }
        }

        m -= shift;  // (what the weights are relative to)
        // join the waves: a common maximum, then the sum of the rescaled parts
        l += __shfl_xor(l, 16, kWave);
        l += __shfl_xor(l, 32, kWave);
        if (g == 0) sm[wave * 16 + c] = m;
        __syncthreads();
        float mx = sm[c];
#pragma unroll
        for (int w = 1; w < NW; ++w) mx = fmaxf(mx, sm[w * 16 + c]);
        // (no maximum: the wave has seen nothing, its sums are zeros, or nothing but NaN)
        const float f = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - mx);
        if (g == 0) sl[wave * 16 + c] = l * f;
        if constexpr (PACK) {
#pragma unroll
            for (int e = 0; e < VD; ++e)
#pragma unroll
                for (int r = 0; r < 4; ++r) o[e][r] = sum_columns<kGroup>(o[e][r]);
        }
        if (c < rows) {
            float *to = join + (wave * hd.rows + c) * kRow + g * 4 * VD;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int e = 0; e < VD; e += 4)
                    *reinterpret_cast<float4 *>(to + r * VD + e) =
                        float4{o[e][r] * f, o[e + 1][r] * f, o[e + 2][r] * f, o[e + 3][r] * f};
        }
        __syncthreads();
        const bool whole = u0 == 0 && u1 == units;
        if (SPLIT && u0 == 0 && u1 < units) mark = KvSplitPair{b, cur.h, mark.flags | kStarts};
        if (SPLIT && u0 > 0 && u1 == units) mark.flags |= kEnds;
        const KvPartial part_ws(a, hd, DP, (int64_t)blockIdx.x * 2 + (u0 == 0));
        int first = threadIdx.x;  // (opaque: its addresses stay out of the loop's registers)
        asm volatile("" : "+v"(first));
        for (int at = first; at < rows * (DP / 4); at += NW * 64) {
            const int r = at / (DP / 4), d = at % (DP / 4) * 4;
            float mr = sm[r];
#pragma unroll
            for (int w = 1; w < NW; ++w) mr = fmaxf(mr, sm[w * 16 + r]);
            float lr = 0.0f;
            float4 y = {};
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                lr += sl[w * 16 + r];
                const float4 z =
                    *reinterpret_cast<const float4 *>(join + (w * hd.rows + r) * kRow + d);
                y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
            }
            if (SPLIT && !whole) {
                *reinterpret_cast<float4 *>(part_ws.o + r * DP + d) = y;
                if (d == 0) part_ws.m[r] = mr, part_ws.l[r] = lr;
            } else if (d < D) {
                store_out<FP32>(a.out, (b * a.hq + (int64_t)kvh * hd.group + part * 16 + r) * D + d,
                                y, lr);
            }
        }
        __syncthreads();
        if (!SPLIT) break;
        cur.left -= end - cur.at;
        cur.at = 0;
        if (++cur.h == hd.count) cur.h = 0, ++cur.b;
    }
    if (SPLIT && threadIdx.x == 0) reinterpret_cast<KvSplitPair *>(a.ws)[blockIdx.x] = mark;
}

// Joins the parts of the pair that workgroup blockIdx.x of the split kernel
// started and others went on with, in the workgroups' order.
template <int DP, bool FP32>
__global__ __launch_bounds__(256) void k_kv_decode_join(KvAttnArgs a) {
    const KvHeads hd(a);
    const KvSplitPair *marks = reinterpret_cast<const KvSplitPair *>(a.ws);
    const KvSplitPair sp = marks[blockIdx.x];
    if (!(sp.flags & kStarts)) return;
    int parts = 1;  // up to the workgroup with the pair's last units
    for (int k = blockIdx.x + 1; k < kSplitBlocks; k += kWave) {
        const int kk = k + threadIdx.x % kWave;
        const uint64_t hit = __ballot(kk < kSplitBlocks && marks[kk].flags & kEnds);
        parts += hit ? __ffsll((unsigned long long)hit) : kWave;
        if (hit) break;
    }
    const int64_t b = sp.b;
    const int kvh = sp.h / hd.per_head, part = sp.h % hd.per_head, D = a.c.D, r = blockIdx.y;
    if (r >= min(hd.group - part * 16, 16)) return;
    // DP / 4 threads have a row's values, 4 each; kGroups of them take parts in turn
    constexpr int kLanes = DP / 4, kGroups = 256 / kLanes;
    __shared__ float4 so[kGroups][kLanes];
    __shared__ float sm[kGroups], sl[kGroups];
    const int grp = threadIdx.x / kLanes, d = threadIdx.x % kLanes * 4;
    float m = -INFINITY, l = 0.0f;
    float4 y = {};
    for (int i = grp; i < parts; i += kGroups) {
        const KvPartial p(a, hd, DP, ((int64_t)blockIdx.x + i) * 2 + (i == 0));
        add_part(m, l, y, p.m[r], p.l[r], *reinterpret_cast<const float4 *>(p.o + r * DP + d));
    }
    so[grp][threadIdx.x % kLanes] = y;
    if (d == 0) sm[grp] = m, sl[grp] = l;
    __syncthreads();
    if (grp != 0 || d >= D) return;
#pragma unroll
    for (int i = 1; i < kGroups; ++i) add_part(m, l, y, sm[i], sl[i], so[i][threadIdx.x % kLanes]);
    store_out<FP32>(a.out, (b * a.hq + (int64_t)kvh * hd.group + part * 16 + r) * D + d, y, l);
}

namespace {

// Up to so many tokens (of a table's row, or visible in the window) a pair is one
// workgroup's; longer ones are split and joined by a second launch.  us, whole / split,
// equally long sequences, 4 query heads a cache head of 128, bf16:
//   pairs    512 tokens    1024          2048           4096
//      1      6.5 /  9.4    8.9 /  9.8    13.5 /  10.1   22.3 /  11.0
//     64      6.9 / 11.9   11.0 / 14.5    23.4 /  21.0   43.3 /  29.4
//    256     11.6 / 17.5   22.1 / 28.9    42.4 /  48.0   81.9 /  87.8
//   1024     47.8 / 50.3   85.6 / 93.0   160.9 / 172.7  318.4 / 334.0
// The host knows the table's width, not the lengths: where a row is half full, the
// column to its left decides.
constexpr int64_t kWholeTokens = 2048;

template <int DP, bool INT8>
size_t lds_bytes(int waves, int rows) {
    const int join = rows * (DP + 4) * 4, stage = 16 * DP * (INT8 ? 1 : 2);
    return (size_t)waves * (std::max(join, stage) + 2 * 16 * 4);
}

template <int DP, bool INT8, bool FP32, bool PACK>
hipError_t launch_dp(const KvAttnArgs &a, const char **path, hipStream_t st) {
    const KvHeads hd(a);
    const int64_t pairs = a.B * hd.count;
    // Tokens of the longest sequence that the table can hold and the window shows
    int64_t most = a.c.W << a.c.shift;
    if (a.window) most = std::min<int64_t>(most, (int64_t)a.window + a.sinks + 64);
    if (most <= kWholeTokens) {
        constexpr int kWholeWaves = DP == 256 && FP32 && !PACK ? 4 : 8;  // (registers)
        const size_t lds = lds_bytes<DP, INT8>(kWholeWaves, hd.rows);
        auto *k = k_kv_decode<DP, INT8, FP32, PACK, kWholeWaves, false>;
        *path = "kv_decode";
        launch_kv(k, dim3((unsigned)pairs), dim3(kWholeWaves * 64), lds, st, a);
    } else {
        const size_t lds = lds_bytes<DP, INT8>(kSplitWaves, hd.rows);
        auto *k = k_kv_decode<DP, INT8, FP32, PACK, kSplitWaves, true>;
        *path = "kv_decode_split";
        launch_kv(k, dim3(kSplitBlocks), dim3(kSplitWaves * 64), lds, st, a);
        hipLaunchKernelGGL((k_kv_decode_join<DP, FP32>), dim3(kSplitBlocks, hd.rows), dim3(256), 0,
                           st, a);
    }
    return hipGetLastError();
}

template <int DP, bool INT8, bool FP32>
hipError_t launch_group(const KvAttnArgs &a, const char **path, hipStream_t st) {
    return a.hq / a.c.heads <= (FP32 ? 4 : 8) ? launch_dp<DP, INT8, FP32, true>(a, path, st)
                                              : launch_dp<DP, INT8, FP32, false>(a, path, st);
}

template <int DP>
hipError_t launch_types(const KvAttnArgs &a, const char **path, hipStream_t st) {
    if (a.int8)
        return a.fp32 ? launch_group<DP, true, true>(a, path, st) : launch_group<DP, true, false>(a, path, st);
    return a.fp32 ? launch_group<DP, false, true>(a, path, st) : launch_group<DP, false, false>(a, path, st);
}

}  // namespace

size_t kv_decode_ws_bytes(int64_t hq, int64_t heads, int64_t D) {
    const int64_t rows = std::min<int64_t>(hq / heads, 16);
    const int64_t DP = D <= 64 ? 64 : D <= 128 ? 128 : 256;
    return (size_t)(kSplitBlocks * (16 + 2 * rows * (DP + 4) * 4));
}

hipError_t launch_kv_decode(const KvAttnArgs &a, const char **path, hipStream_t st) {
    return a.c.D <= 64 ? launch_types<64>(a, path, st)
           : a.c.D <= 128 ? launch_types<128>(a, path, st)
                          : launch_types<256>(a, path, st);
}

}  // namespace w4
