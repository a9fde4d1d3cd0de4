// Low-rank adapters beside a shared product:
//   Y[m] += scale_a ((X[m] A_a^T) B_a^T), a = ids[m].
// Two launches: S = X A^T into the workspace, in parts of K, then Y += scale S B^T.
//
// Rows are taken in tiles of 16 or 32 as they lie.  A workgroup goes through the
// different adapters that its tile names (a ballot over the tile's ids; slots of
// workgroups share them out) and computes the tile's rows of one adapter at a
// time, so that no plan, no sorting and no atomics are needed and a row's result
// does not depend on its neighbours (but on M: with it change the parts of K, whose
// sums are added in their order).
//
// Products are bf16 MFMAs (16 x 16 x 32) with fp32 sums.  An fp32 value of X, and
// every value of S, is three bf16 terms of 8 bits each, cut off one after the
// other: they hold its 24 bits exactly (down to 2^-110: the matrix cores take
// subnormal terms, whose last bit is 2^-133), and the largest values do not round up to
// infinity.  What is left of an infinity is NaN, and so are its products (its first
// term alone would take a test of every value: 8192 rows of 4096 fp32, rank 64 and 128,
// first launch 52 -> 55 and 92 -> 97 us, second 62 -> 62 and 116 -> 119).
#include <algorithm>
#include <type_traits>

#include "kv_common.h"
#include "layer.h"

namespace w4 {

template <int N> using Int = std::integral_constant<int, N>;

struct LoraPlan {
    int slots, splits, kc;  // workgroups of a tile, parts of K, length of a part
    int rp;                 // rank, rounded up to 16: a row of S
    int tiles;
    int nc;                 // channels of a workgroup of the second launch
};

// ------------------------------------------------------------------ helpers
// (uniform: the loops of a wave then run on scalars)
__device__ __forceinline__ int wave_id() {
    return __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
}

// The adapter of a row, or -1.
__device__ __forceinline__ int lora_id(const LoraArgs &a, int64_t m) {
    const int id = m < a.M ? a.ids[m] : -1;
    return (uint32_t)id < (uint32_t)a.adapters ? id : -1;
}

__device__ __forceinline__ int lora_rank(const LoraArgs &a, int id) {
    return a.ranks ? min(max(a.ranks[id], 0), a.rank) : a.rank;
}

// f(adapter, mask of its rows) for every slots-th different adapter of the tile
// whose ids the lanes hold.
template <typename F>
__device__ __forceinline__ void each_adapter(int id, int slot, int slots, F f) {
    uint64_t todo = __ballot(id >= 0);
    for (int i = 0; todo; ++i) {
        const int cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
        const uint64_t match = __ballot(id == cur);
        todo &= ~match;
        if (i % slots == slot) f(cur, match);
    }
}

// Eight floats as three bf16 terms, each the upper half of what is left.
__device__ __forceinline__ void cut3(const float (&f)[8], v8bf (&out)[3]) {
    uint32_t r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = __float_as_uint(f[j]);
#pragma unroll
    for (int t = 0; t < 3; ++t) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __builtin_amdgcn_perm(r[2 * j + 1], r[2 * j], 0x07060302u);
        out[t] = __builtin_bit_cast(v8bf, uint4{w[0], w[1], w[2], w[3]});
        if (t < 2) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                r[j] = __float_as_uint(__uint_as_float(r[j]) - __uint_as_float(r[j] & 0xFFFF0000u));
        }
    }
}

// Which of eight bf16 to keep, the first `n` (the others may hold anything).
__device__ __forceinline__ uint4 keep8(int n) {
    auto two = [&](int i) { return n > i + 1 ? ~0u : n > i ? 0xFFFFu : 0u; };
    return uint4{two(0), two(2), two(4), two(6)};
}

__device__ __forceinline__ uint4 and8(uint4 w, uint4 k) {
    return uint4{w.x & k.x, w.y & k.y, w.z & k.z, w.w & k.w};
}

__device__ __forceinline__ uint4 not8(uint4 k) { return uint4{~k.x, ~k.y, ~k.z, ~k.w}; }

// Eight bf16 at an offset that is aligned to 2 bytes; zeros outside the range.
__device__ __forceinline__ uint4 bload8x2(__amdgpu_buffer_rsrc_t r, int off) {
    uint32_t f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __builtin_amdgcn_raw_buffer_load_b16(r, off + 2 * j, 0, 0);
    return uint4{f[0] | f[1] << 16, f[2] | f[3] << 16, f[4] | f[5] << 16, f[6] | f[7] << 16};
}

// Eight values of X, or of A, as operand terms: from p, aligned to its elements, or
// values k, k + 1, ... of a row of `end` (1 or more) and zeros beyond it; no load is in
// a branch.
template <bool FP32> struct Chunk;
template <> struct Chunk<true> {
    float4 a, b;
    __device__ __forceinline__ void whole(const float *p) {
        __builtin_memcpy(&a, p, 16);
        __builtin_memcpy(&b, p + 4, 16);
    }
    __device__ __forceinline__ void some(const float *row, int k, int end) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = row[min(k + j, end - 1)];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = k + j < end ? f[j] : 0.0f;
        a = float4{f[0], f[1], f[2], f[3]}, b = float4{f[4], f[5], f[6], f[7]};
    }
    __device__ __forceinline__ void terms(v8bf (&out)[3]) const {
        const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        cut3(f, out);
    }
};
template <> struct Chunk<false> {
    uint4 w;
    __device__ __forceinline__ void whole(const uint16_t *p) { __builtin_memcpy(&w, p, 16); }
    __device__ __forceinline__ void some(const uint16_t *row, int k, int end) {
        uint32_t f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = row[min(k + j, end - 1)];
        w = and8(uint4{f[0] | f[1] << 16, f[2] | f[3] << 16, f[4] | f[5] << 16, f[6] | f[7] << 16},
                 keep8(end - k));
    }
    __device__ __forceinline__ void terms(v8bf (&out)[1]) const { out[0] = __builtin_bit_cast(v8bf, w); }
};

__device__ __forceinline__ v4f mfma(v8bf a, v8bf b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// ------------------------------------------------------------------ X A^T
// The four waves' sums into this part's rows of S.
template <int MT, int RC>
__device__ __forceinline__ void write_sums(const LoraArgs &a, const LoraPlan &p,
                                           const v4f (*red)[MT * RC][kWave], int64_t m0, int r0,
                                           uint64_t match) {
    for (int i = threadIdx.x; i < MT * RC * kWave; i += 256) {
        const int tc = i / kWave, m = 16 * (tc / RC) + i % 16;
        const int j = r0 + 16 * (tc % RC) + i % kWave / 16 * 4;
        if (!(match >> m & 1) || j >= p.rp) continue;
        v4f s = red[0][tc][i % kWave];
#pragma unroll
        for (int v = 1; v < 4; ++v) s += red[v][tc][i % kWave];
        *reinterpret_cast<v4f *>(a.ws + ((int64_t)blockIdx.x * a.M + m0 + m) * p.rp + j) = s;
    }
}

// Workgroup (tile and slot, part of K, 16 RC rows of A): its four waves take a
// quarter of the part each and add their sums in LDS.  A is the first operand
// and X the second, so that a lane ends with four neighbouring values of a row
// of S.  X is read once (for every 16 RC ranks), straight into registers: this form
// takes every size and alignment: whole steps of 32 k by loads aligned to elements, a
// last one value by value, with no branch between the loads (409 rows of 451, rank 29:
// 6.8 us, with branches 7.9).
template <bool FP32, int MT, int RC>
__global__ __launch_bounds__(256) void k_lora_down(LoraArgs a, LoraPlan p) {
    constexpr int U = FP32 ? 4 / MT : MT * RC >= 8 ? 1 : 8 / (MT * RC);  // k-steps in flight
    constexpr int kTerms = FP32 ? 3 : 1;
    using X = std::conditional_t<FP32, float, uint16_t>;
    __shared__ v4f red[4][MT * RC][kWave];
    const int lane = threadIdx.x % kWave, wave = wave_id();
    const int c16 = lane % 16, q8 = lane / 16 * 8;
    const int K = (int)a.K, r0 = blockIdx.z * (16 * RC);
    const int kw = p.kc / 4, k0 = blockIdx.x * p.kc + wave * kw, k1 = min(k0 + kw, K);
    for (uint32_t tile = blockIdx.y; tile < (uint32_t)(p.tiles * p.slots); tile += gridDim.y) {
        const int64_t m0 = (int64_t)(tile % (uint32_t)p.tiles) * (16 * MT);
        const int id = lane < 16 * MT ? lora_id(a, m0 + lane) : -1;
        const X *rows = reinterpret_cast<const X *>(a.X) + m0 * a.ldx;
        each_adapter(id, (int)(tile / (uint32_t)p.tiles), p.slots, [&](int cur, uint64_t match) {
            const int rank = lora_rank(a, cur);
            if (r0 >= rank) return;
            const int ranks = min(rank - r0, 16 * RC);
            const uint16_t *A = a.A + ((int64_t)cur * a.rank + r0) * a.K;
            // (a lane without a row of X or of A reads the first one: what comes of it is no
            // row's, or is dropped)
            const X *x[MT];
            const uint16_t *w[RC];
            v4f acc[MT][RC];
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                x[t] = rows + (match >> (16 * t + c16) & 1 ? 16 * t + c16 : 0) * a.ldx;
#pragma unroll
                for (int c = 0; c < RC; ++c) acc[t][c] = v4f{0.f, 0.f, 0.f, 0.f};
            }
#pragma unroll
            for (int c = 0; c < RC; ++c)
                w[c] = A + (int64_t)(16 * c + c16 < ranks ? 16 * c + c16 : 0) * K;
            // `steps` k-steps from k; whole: all of their values are the part's
            auto add = [&](int k, auto steps, auto whole) {
                constexpr int kSteps = decltype(steps)::value;
                Chunk<FP32> xs[kSteps][MT];
                Chunk<false> ws[kSteps][RC];
                auto load = [&](auto &chunk, auto *row, int at) {
                    if constexpr (decltype(whole)::value) chunk.whole(row + at);
                    else chunk.some(row, at, k1);
                };
#pragma unroll
                for (int u = 0; u < kSteps; ++u)
#pragma unroll
                    for (int c = 0; c < RC; ++c) load(ws[u][c], w[c], k + 32 * u + q8);
#pragma unroll
                for (int u = 0; u < kSteps; ++u)
#pragma unroll
                    for (int t = 0; t < MT; ++t) load(xs[u][t], x[t], k + 32 * u + q8);
#pragma unroll
                for (int u = 0; u < kSteps; ++u)
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        v8bf f[kTerms];
                        xs[u][t].terms(f);
#pragma unroll
                        for (int c = 0; c < RC; ++c)
#pragma unroll
                            for (int i = kTerms - 1; i >= 0; --i)
                                acc[t][c] = mfma(__builtin_bit_cast(v8bf, ws[u][c].w), f[i], acc[t][c]);
                    }
            };
            int k = k0;
            for (; k + 32 * U <= k1; k += 32 * U) add(k, Int<U>{}, std::true_type{});
            for (; k + 32 <= k1; k += 32) add(k, Int<1>{}, std::true_type{});
            if (k < k1) add(k, Int<1>{}, std::false_type{});
            lds_barrier();  // (the sums of the adapter before have been read)
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int c = 0; c < RC; ++c) red[wave][t * RC + c][lane] = acc[t][c];
            lds_barrier();
            write_sums<MT, RC>(a, p, red, m0, r0, match);
        });
    }
}

// The same for aligned operands: stages of 128 k go through LDS by direct loads,
// whole row pieces of 256 and 512 bytes side by side, since the operands' own layout
// (neighbouring lanes, different rows) costs the address unit four times the cycles
// (8192 rows, K 4096, rank 32, 134 MB: 35 us, 45 straight into registers).  X goes past
// the caches, whose place A has (35 us, 38 through them).  16-byte pieces of a row are
// stored at their index xor the row, so that 16 rows' reads of one piece hit all
// banks.  Wave w takes k-step w of each stage; three stages, two of them in flight
// (two slots 34 us, four 48, for want of a second workgroup).
template <bool FP32, int MT, int RC>
__global__ __launch_bounds__(256) void k_lora_down_lds(LoraArgs a, LoraPlan p) {
    constexpr int kTerms = FP32 ? 3 : 1;
    constexpr int kStage = 128, kSlots = 3;
    constexpr int kXRow = kStage * (FP32 ? 4 : 2), kARow = kStage * 2;  // bytes
    constexpr int kXBytes = 16 * MT * kXRow, kBytes = kXBytes + 16 * RC * kARow;
    constexpr int kXLoads = kXBytes / 4096, kALoads = RC;  // 1 KB loads of a wave and stage
    constexpr int kLoads = kXLoads + kALoads;
    __shared__ __align__(1024) uint8_t lds[kSlots * kBytes];
    static_assert(4 * MT * RC * 1024 <= kSlots * kBytes, "the sums fit the stages' memory");
    const int lane = threadIdx.x % kWave, wave = wave_id();
    const int c16 = lane % 16, q = lane / 16;
    const int K = (int)a.K, r0 = blockIdx.z * (16 * RC);
    const int k0 = blockIdx.x * p.kc, k1 = min(k0 + p.kc, K);
    const uint32_t base = lds_addr(lds);
    for (uint32_t tile = blockIdx.y; tile < (uint32_t)(p.tiles * p.slots); tile += gridDim.y) {
        const int64_t m0 = (int64_t)(tile % (uint32_t)p.tiles) * (16 * MT);
        const int id = lane < 16 * MT ? lora_id(a, m0 + lane) : -1;
        const v4i rx = buffer_desc(reinterpret_cast<const uint8_t *>(a.X) + m0 * a.ldx * (FP32 ? 4 : 2),
                                   kMaxRange);
        each_adapter(id, (int)(tile / (uint32_t)p.tiles), p.slots, [&](int cur, uint64_t match) {
            const int rank = lora_rank(a, cur);
            if (r0 >= rank) return;
            const int ranks = min(rank - r0, 16 * RC);
            const v4i ra = buffer_desc(a.A + ((int64_t)cur * a.rank + r0) * a.K,
                                       (int64_t)ranks * a.K * 2);
            // this lane's piece of each of the wave's loads: byte offset at k = 0, and its k
            constexpr int kXPieces = kXRow / 16, kAPieces = kARow / 16;
            int xoff[kXLoads], xk[kXLoads], aoff[kALoads], ak[kALoads];
#pragma unroll
            for (int i = 0; i < kXLoads; ++i) {
                const int n = (wave * kXLoads + i) * kWave + lane, m = n / kXPieces;
                xk[i] = ((n % kXPieces) ^ (m % 16)) * (FP32 ? 4 : 8);
                xoff[i] = match >> m & 1 ? (int)(m * a.ldx + xk[i]) * (FP32 ? 4 : 2) : kOOB;
            }
#pragma unroll
            for (int i = 0; i < kALoads; ++i) {
                const int n = (wave * kALoads + i) * kWave + lane, j = n / kAPieces;
                ak[i] = ((n % kAPieces) ^ (j % 16)) * 8;
                aoff[i] = j < ranks ? (j * K + ak[i]) * 2 : kOOB;
            }
            auto fetch = [&](int k, int slot) {
                const uint32_t to = base + slot * kBytes;
#pragma unroll
                for (int i = 0; i < kXLoads; ++i)
                    dma16_nt(rx, to + (wave * kXLoads + i) * 1024,
                          k + xk[i] < k1 && xoff[i] != kOOB ? xoff[i] + k * (FP32 ? 4 : 2) : kOOB, 0);
#pragma unroll
                for (int i = 0; i < kALoads; ++i)
                    dma16(ra, to + kXBytes + (wave * kALoads + i) * 1024,
                          k + ak[i] < k1 && aoff[i] != kOOB ? aoff[i] + k * 2 : kOOB, 0);
            };
            v4f acc[MT][RC];
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int c = 0; c < RC; ++c) acc[t][c] = v4f{0.f, 0.f, 0.f, 0.f};
            wait_and_barrier<0>();  // (LDS is free, and no store is counted among the loads)
            fetch(k0, 0);
            if (k0 + kStage < k1) fetch(k0 + kStage, 1);
            int slot = 0;
            for (int k = k0; k < k1; k += kStage) {
                if (k + kStage < k1) wait_and_barrier<kLoads>();
                else wait_and_barrier<0>();
                if (k + 2 * kStage < k1) fetch(k + 2 * kStage, slot == 0 ? 2 : slot - 1);
                const uint8_t *from = lds + slot * kBytes;
                const int kk = k + 32 * wave + 8 * q;
                uint4 w[RC];
#pragma unroll
                for (int c = 0; c < RC; ++c) {
                    w[c] = *reinterpret_cast<const uint4 *>(from + kXBytes + (16 * c + c16) * kARow +
                                                            ((4 * wave + q) ^ c16) * 16);
                    if (kk >= k1) w[c] = uint4{};
                }
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const uint8_t *row = from + (16 * t + c16) * kXRow;
                    Chunk<FP32> x;
                    if constexpr (FP32) {
                        x.a = *reinterpret_cast<const float4 *>(row + ((8 * wave + 2 * q) ^ c16) * 16);
                        x.b = *reinterpret_cast<const float4 *>(row + ((8 * wave + 2 * q + 1) ^ c16) * 16);
                    } else {
                        x.w = *reinterpret_cast<const uint4 *>(row + ((4 * wave + q) ^ c16) * 16);
                    }
                    if (kk >= k1) x = Chunk<FP32>{};
                    v8bf f[kTerms];
                    x.terms(f);
#pragma unroll
                    for (int c = 0; c < RC; ++c)
#pragma unroll
                        for (int i = kTerms - 1; i >= 0; --i)
                            acc[t][c] = mfma(__builtin_bit_cast(v8bf, w[c]), f[i], acc[t][c]);
                }
                slot = slot == kSlots - 1 ? 0 : slot + 1;
            }
            v4f(*red)[MT * RC][kWave] = reinterpret_cast<v4f(*)[MT * RC][kWave]>(lds);
            lds_barrier();  // (every wave has read its last stage)
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int c = 0; c < RC; ++c) red[wave][t * RC + c][lane] = acc[t][c];
            lds_barrier();
            write_sums<MT, RC>(a, p, red, m0, r0, match);
        });
    }
}

// ------------------------------------------------------------------ Y += S B^T
// Workgroup (tile and slot, nc channels).  The parts of S are added in order into
// LDS once; a wave keeps the terms of its rows in registers while it goes through
// 64 channels of B at a time (B is the first operand: a lane has four neighbouring
// channels of a row).  The 256 channels of the four waves change lanes in LDS, so
// that Y is read and written in whole pieces of 1 KB of a row, and only its own rows;
// in tiles of 32 rows, those of prompts, past the caches (8192 rows, K = N = 4096,
// rank 32, both launches: 90 -> 85 us).  Without VEC, B's pieces may lie anywhere (16
// rows -> 28671, rank 61: 20.4 us, 13.5 where aligned; value by value 44).
template <bool VEC, bool YVEC, int MT, int KS>
__global__ __launch_bounds__(256) void k_lora_up(LoraArgs a, LoraPlan p) {
    constexpr int NU = 4;  // blocks of 16 channels whose loads are in flight
    constexpr int kRow = 32 * KS + 4;
    __shared__ __align__(16) float S[16 * MT][kRow];
    __shared__ __align__(16) float D[16 * MT][260];
    const int lane = threadIdx.x % kWave, wave = wave_id();
    const int c16 = lane % 16, q = lane / 16;
    const int64_t n0 = (int64_t)blockIdx.x * p.nc;
    const int len = (int)min((int64_t)p.nc, a.N - n0);
    for (uint32_t tile = blockIdx.y; tile < (uint32_t)(p.tiles * p.slots); tile += gridDim.y) {
        const int64_t m0 = (int64_t)(tile % (uint32_t)p.tiles) * (16 * MT);
        const int id = lane < 16 * MT ? lora_id(a, m0 + lane) : -1;
        float *rows = a.Y + m0 * a.ldy + n0;
        each_adapter(id, (int)(tile / (uint32_t)p.tiles), p.slots, [&](int cur, uint64_t match) {
            const int rank = lora_rank(a, cur);
            const float scale = a.scales ? a.scales[cur] : 1.0f;
            const uint16_t *B = a.B + ((int64_t)cur * a.N + n0) * a.rank;
            const auto rb = make_rsrc(B, (int64_t)len * a.rank * 2);  // (beyond it: zeros)
            // This lane's ranks of step s: 32 s + 8 q and the 7 behind it.  Where pieces may not
            // be aligned, a row's last piece is the 8 that end it, of which those that an
            // earlier piece has are dropped, so that every load is whole and within its row.
            int first[KS], at[KS];  // rank of a piece's first value; its bytes in a block of 16 channels
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const int j = 32 * s + 8 * q;
                first[s] = VEC || a.rank < 8 ? j : min(j, a.rank - 8);
                // (the pool's rank, so that no load waits for the adapter's own)
                at[s] = j < a.rank ? (c16 * a.rank + j) * 2 : kOOB;
            }
            uint4 w[NU][KS];
            v4f y[4 * MT];  // of rows wave, wave + 4, ...: this lane's four channels of 256
            auto load_b = [&](int n, auto load) {
#pragma unroll
                for (int u = 0; u < NU; ++u)
#pragma unroll
                    for (int s = 0; s < KS; ++s) w[u][s] = load(n + 64 * wave + 16 * u, s);
            };
            auto load_channels = [&](int n) {
                auto offset = [&](int ch, int s) { return (int)((uint32_t)at[s] + (uint32_t)(ch * a.rank * 2)); };
                if constexpr (VEC) {
                    load_b(n, [&](int ch, int s) { return bload16(rb, offset(ch, s)); });
                } else if (a.rank >= 8) {
                    load_b(n, [&](int ch, int s) {
                        uint4 v;
                        __builtin_memcpy(&v, B + min(ch + c16, len - 1) * a.rank + first[s], 16);
                        return v;
                    });
                } else {
                    load_b(n, [&](int ch, int s) { return bload8x2(rb, offset(ch, s)); });
                }
            };
            // this lane's channels: 4 lane + e, or lane + 64 e where Y goes value by value
            auto channel = [&](int e) { return YVEC ? 4 * lane + e : lane + 64 * e; };
            auto each_y = [&](int n, auto f) {
#pragma unroll
                for (int i = 0; i < 4 * MT; ++i) {
                    const int m = wave + 4 * i;
                    if (!(match >> m & 1)) continue;
                    float *at = rows + m * a.ldy + n;
                    if constexpr (YVEC) {
                        v4f *own = reinterpret_cast<v4f *>(at + 4 * lane);
                        if (n + 4 * lane < len)
                            f(i, m, [&](v4f &v) { v = MT > 1 ? __builtin_nontemporal_load(own) : *own; },
                              [&](const v4f &v) {
                                  if constexpr (MT > 1) __builtin_nontemporal_store(v, own);
                                  else *own = v;
                              });
                    } else {
                        f(i, m,
                          [&](v4f &v) {
#pragma unroll
                              for (int e = 0; e < 4; ++e)
                                  if (n + channel(e) < len) v[e] = at[channel(e)];
                          },
                          [&](const v4f &v) {
#pragma unroll
                              for (int e = 0; e < 4; ++e)
                                  if (n + channel(e) < len) at[channel(e)] = v[e];
                          });
                    }
                }
            };
            auto read = [&](int i, int, auto get, auto) { get(y[i]); };
            int n = 0;
            load_channels(n);  // (in flight while S is summed)
            each_y(n, read);
            if (rank == 0) return;
            uint4 keep[KS];  // which values of a lane's pieces count
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                keep[s] = keep8(rank - first[s]);
                if constexpr (!VEC) keep[s] = and8(keep[s], not8(keep8(32 * s + 8 * q - first[s])));
            }
            lds_barrier();  // (the rows of the adapter before have been read)
            const int64_t part = a.M * p.rp;
            for (int i = threadIdx.x; i < 16 * MT * 8 * KS; i += 256) {
                const int m = i / (8 * KS), j = i % (8 * KS) * 4;
                v4f s = v4f{0.f, 0.f, 0.f, 0.f};
                if ((match >> m & 1) && j < rank) {
                    const float *src = a.ws + (m0 + m) * p.rp + j;
                    for (int k = 0; k < p.splits; k += 8) {  // (eight parts' loads at a time)
                        v4f v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (k + e < p.splits)
                                v[e] = *reinterpret_cast<const v4f *>(src + (k + e) * part);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (k + e < p.splits) s += v[e];
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[e] = j + e < rank ? s[e] : 0.0f;
                }
                *reinterpret_cast<v4f *>(&S[m][j]) = s;
            }
            lds_barrier();
            v8bf f[MT][KS][3];
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    float v[8];
                    const float *src = &S[16 * t + c16][first[s]];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = VEC || first[s] + e >= 32 * s + 8 * q ? src[e] : 0.0f;
                    cut3(v, f[t][s]);
                }
            for (;;) {
                const int next = n + 64 * NU;
#pragma unroll
                for (int u = 0; u < NU; ++u)
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        v4f acc = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int s = 0; s < KS; ++s)
#pragma unroll
                            for (int i = 2; i >= 0; --i)
                                acc = mfma(__builtin_bit_cast(v8bf, and8(w[u][s], keep[s])), f[t][s][i], acc);
                        *reinterpret_cast<v4f *>(&D[16 * t + c16][64 * wave + 16 * u + 4 * q]) = acc;
                    }
                if (next < len) load_channels(next);
                lds_barrier();
                each_y(n, [&](int i, int m, auto, auto put) {
                    v4f v;
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(scale, D[m][channel(e)], y[i][e]);
                    put(v);
                });
                if (next >= len) break;
                n = next;
                each_y(n, read);
                lds_barrier();  // (D has been read)
            }
        });
    }
}

// ------------------------------------------------------------------ launches
constexpr int kMaxSplits = 16;
constexpr int64_t kSplitRows = 32768;  // rows of S in the workspace beyond the first part, at most

// A tile's 32 rows lie within a descriptor's range.
constexpr int64_t kMaxStride = (int64_t)1 << 23;

static int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }

// S in up to 1 + min(15, 32768 / M) parts: the size grows with M and rank alone.
size_t lora_ws_bytes(int64_t M, int64_t, int64_t, int64_t rank) {
    const int64_t rows = M + std::min(M * (kMaxSplits - 1), kSplitRows);
    return (size_t)rows * (size_t)round16(rank) * 4;
}

template <bool FP32, int MT, int RC>
static void go_down_as(const LoraArgs &a, const LoraPlan &p, bool vec, hipStream_t st) {
    const dim3 g((unsigned)p.splits, (unsigned)std::min<int64_t>((int64_t)p.tiles * p.slots, 65535),
                 (unsigned)((a.rank + 16 * RC - 1) / (16 * RC)));
    if (vec) launch_kv(k_lora_down_lds<FP32, MT, RC>, g, dim3(256), 0, st, a, p);
    else launch_kv(k_lora_down<FP32, MT, RC>, g, dim3(256), 0, st, a, p);
}

template <bool FP32, int MT>
static void go_down(const LoraArgs &a, const LoraPlan &p, bool vec, hipStream_t st) {
    if (a.rank <= 16) go_down_as<FP32, MT, 1>(a, p, vec, st);
    else if (a.rank <= 32) go_down_as<FP32, MT, 2>(a, p, vec, st);
    else go_down_as<FP32, MT, 4>(a, p, vec, st);
}

template <bool VEC, bool YVEC, int MT>
static void go_up(const LoraArgs &a, const LoraPlan &p, hipStream_t st) {
    const dim3 g((unsigned)((a.N + p.nc - 1) / p.nc), (unsigned)std::min<int64_t>((int64_t)p.tiles * p.slots, 65535));
    if (a.rank <= 32) launch_kv(k_lora_up<VEC, YVEC, MT, 1>, g, dim3(256), 0, st, a, p);
    else if (a.rank <= 64) launch_kv(k_lora_up<VEC, YVEC, MT, 2>, g, dim3(256), 0, st, a, p);
    else if (a.rank <= 128) launch_kv(k_lora_up<VEC, YVEC, MT, 4>, g, dim3(256), 0, st, a, p);
    else if constexpr (MT == 1) launch_kv(k_lora_up<VEC, YVEC, 1, 8>, g, dim3(256), 0, st, a, p);
}

template <int MT>
static void go(const LoraArgs &a, const char **path, hipStream_t st) {
    auto at16 = [](const void *q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
    const int64_t tiles = (a.M + 16 * MT - 1) / (16 * MT);
    // Workgroups of a tile: as many as its adapters can use, or 2048 of the call.  Their
    // index is the slowest: beside the tile's, the idle ones of prompts (one adapter a
    // tile) left half of the XCDs without work (first launch of 8192 rows 53 us, 45).
    auto slots = [&](int64_t others) {
        const int64_t most = std::min<int64_t>(16 * MT, a.adapters);
        return (int)std::max<int64_t>(1, std::min<int64_t>(most, 2048 / std::max<int64_t>(1, others)));
    };
    LoraPlan p{};
    p.rp = (int)round16(a.rank);
    // Parts of K of 512 or more (64 rows, K 4096, us for 2 / 4 / 8 / 16 parts: 9.1 / 6.4 / 5.4 /
    // 6.1), fewer where the tiles fill the GPU (8192 rows, both launches, 2 / 4 / 8: 92 / 85 / 87).
    int64_t splits = std::min<int64_t>(1 + std::min<int64_t>(kMaxSplits - 1, kSplitRows / a.M),
                                       std::min<int64_t>((a.K + 511) / 512, (1024 + tiles - 1) / tiles));
    p.kc = (int)(((a.K + splits - 1) / splits + 127) / 128 * 128);
    p.splits = (int)((a.K + p.kc - 1) / p.kc);
    p.slots = slots(tiles * p.splits);
    p.tiles = (int)tiles;
    const bool xv = a.K % 8 == 0 && at16(a.X) && at16(a.A) && a.ldx * (a.fp32 ? 4 : 2) % 16 == 0 &&
                    a.ldx <= kMaxStride;
    a.fp32 ? go_down<true, MT>(a, p, xv, st) : go_down<false, MT>(a, p, xv, st);

    const bool bv = a.rank % 8 == 0 && at16(a.B);
    const bool yv = a.N % 4 == 0 && a.ldy % 4 == 0 && at16(a.Y);
    // Channels of a workgroup: 256, and more where there are workgroups enough, since each
    // sums S and splits it once (us for 256 / 512 / 1024 / 2048: 64 rows -> 11008, rank 16, 13.8 /
    // 10.7 / 8.6 / 10.0; 16 rows -> 28672, rank 64, 24 / 18 / 13.5 / 13.8; 8192 rows -> 4096, both
    // launches, 90 / 85 / 92; one row -> 6912 3.5 / 3.8 / 4.7).  As many as leave two workgroups
    // a CU, 512 in all: beyond them is another round (16 rows of 16 adapters, rank 64, us for
    // 256 / 512 / 768 / 1024: 544 workgroups of 256 channels 9.3 / 7.1 / 7.6 / 8.4; 1024 11.9 /
    // 7.7 / 9.2 / 9.0; 1056 14.2 / 12.5 / 9.3 / 10.7; 1552 19.5 / 14.3 / 14.5 / 11.9); four a CU
    // in tiles of 32 rows, whose slots mostly find no adapter and end (300 rows, 8 adapters, 640
    // workgroups 4.8 / 7.0, 1280 7.5 / 7.2).
    const int64_t chunks = (a.N + 255) / 256, full = 512 * MT;
    const int64_t work = tiles * std::min<int64_t>(16 * MT, a.adapters) * chunks;
    const int64_t per = std::min<int64_t>(MT == 1 ? 4 : 2, (work + full - 1) / full);
    p.nc = (int)(256 * per);
    p.slots = slots(tiles * ((a.N + p.nc - 1) / p.nc));
    if (bv) yv ? go_up<true, true, MT>(a, p, st) : go_up<true, false, MT>(a, p, st);
    else yv ? go_up<false, true, MT>(a, p, st) : go_up<false, false, MT>(a, p, st);
    // (the operands that are not taken in aligned pieces; X's includes A's)
    static const char *const kPaths[] = {"lora",       "lora_odd_x",  "lora_odd_b",  "lora_odd_xb",
                                         "lora_odd_y", "lora_odd_xy", "lora_odd_by", "lora_odd_xby"};
    *path = kPaths[(xv ? 0 : 1) + (bv ? 0 : 2) + (yv ? 0 : 4)];
}

hipError_t launch_lora(const LoraArgs &a, const char **path, hipStream_t st) {
    // Tiles of 32 rows halve the traffic of A and B, of 16 spread a step's adapters over
    // more workgroups (8192 rows, first launch, 32 / 16: 33 / 37 us); more than 128 ranks
    // of 32 rows would not fit the registers.
    if (a.M <= 256 || a.rank > 128) go<1>(a, path, st);
    else go<2>(a, path, st);
    return hipGetLastError();
}

}  // namespace w4
