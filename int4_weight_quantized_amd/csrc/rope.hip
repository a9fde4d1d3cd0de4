// Rotary positions: a standalone rotation of heads, and one on the way into the
// paged cache (queries rotated, keys rotated and cached, values cached).
// Pair i of a token at position p turns by t = p turns[i] full turns:
//   (a, b) -> (fl(fl(a c) - fl(b s)), fl(fl(b c) + fl(a s))),
//   c, s = fp32 of magnitude * cos, sin(2 pi t).
// Angles are taken in fp64: p turns[i] loses 2^-53 of itself, so that a token at
// position 10^6 still has its angle to 10^-10 where fp32 would be off by a hundredth
// of a turn (0.013 at base 10000, nearly a tenth of a radian), and c and s are rounded
// once.
//
// A wave takes one token: it computes the token's angles (64 at once), keeps those
// of its lanes' values in registers, and goes through the token's heads, 1 KB at a
// time, four loads ahead; waves share nothing.  Calls of few tokens split a
// token's heads over several waves, each with the angles.  Bound by memory (into the
// cache: 6984 tokens of 64 / 8 heads of 128, fp32, 543 MB, 86 us, 6.3 TB/s).
#include <algorithm>
#include <type_traits>

#include "kv_common.h"
#include "layer.h"

namespace w4 {

constexpr int kHalf = 256;  // pairs of a token, at most
constexpr int kAhead = 4;   // loads of a lane in flight

template <int N> using Int = std::integral_constant<int, N>;

// Memory of one wave.
struct RopeLds {
    float2 cs[kHalf];
    float4 swap[kWave * 2];
};

// LDS of a wave is read in the order in which it was written; this keeps the
// compiler to it.
__device__ __forceinline__ void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// The factors of the V values d, d + 1, ... of a head that this lane holds.
template <int V>
struct Turn {
    float c[V], s[V];  // value * c + other * s
    int rot;           // how many of them turn
    int other;         // first value of the partners' 16-byte piece (half layout), or -1
    int d;
};

template <int V>
__device__ __forceinline__ Turn<V> rope_turn(const RopeView &r, int64_t pos, int d, RopeLds &l) {
    for (int i = threadIdx.x % kWave; i < r.half; i += kWave) {
        const double turns = (double)pos * r.turns[i];
        double s, c;
        sincospi(2.0 * (turns - rint(turns)), &s, &c);
        l.cs[i] = float2{(float)(r.magnitude * c), (float)(r.magnitude * s)};
    }
    wave_fence();
    Turn<V> t;
    t.d = d;
    t.rot = r.rot - d;
    t.other = r.half % V == 0 && d < r.rot ? (d < r.half ? d + r.half : d - r.half) : -1;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int e = min(d + j, r.rot - 1);
        const bool low = r.pairs ? e % 2 == 0 : e < r.half;
        const float2 u = l.cs[r.pairs ? e / 2 : low ? e : e - r.half];
        t.c[j] = u.x;
        t.s[j] = low ? -u.y : u.y;
    }
    return t;
}

// Rotate f.  In the half layout the other value of a pair is another lane's of the
// same head, `group` lanes that start at lane `first` of the wave; it goes through LDS.
template <int V>
__device__ __forceinline__ void rotate(const RopeView &r, const Turn<V> &t, int first, float4 *swap,
                                       float (&f)[V]) {
    float o[V];
    if (r.pairs) {
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = f[j ^ 1];
    } else {
        const int lane = threadIdx.x % kWave;
        const float *from = reinterpret_cast<const float *>(swap) + first * V;
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            swap[lane * (V / 4) + i] = float4{f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]};
        wave_fence();
        if (r.half % V == 0) {
            const int at = max(t.other, 0);
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
                const float4 v = *reinterpret_cast<const float4 *>(from + at + 4 * i);
                o[4 * i] = v.x, o[4 * i + 1] = v.y, o[4 * i + 2] = v.z, o[4 * i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int e = min(t.d + j, r.rot - 1);
                o[j] = from[e < r.half ? e + r.half : e - r.half];
            }
        }
        wave_fence();
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float y = f[j] * t.c[j] + o[j] * t.s[j];
        f[j] = j < t.rot ? y : f[j];
    }
}

// How rows are read: a value at a time where an address or a stride is aligned to
// elements only; through the caches where heads end inside a line of 128 bytes, which
// two loads then share; else past them.  (us, past / through: 8191 tokens of 40 heads
// of 128 fp32, output in memory that the last call's had, 51 / 63; in new memory 65 /
// 66; heads of 80 bf16 32 / 29.  The output goes through the caches for the attention
// that reads it, past them 63 in either.)
enum { kSome, kCached, kStream };

// V values of a lane as they lie in memory, so that a load waits for nothing.
template <bool FP32, int V>
struct Raw {
    static constexpr int kSize = FP32 ? 4 : 2, kPieces = V * kSize / 16;
    uint4 w[kPieces];

    // beyond the row's range: zeros
    template <int MODE>
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t at) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            w[i] = MODE == kStream ? bload16_nt(r, (int)(at + 16 * i)) : bload16(r, (int)(at + 16 * i));
    }
    // the same for rows that are aligned to their elements only
    __device__ __forceinline__ void load_some(const void *row, int at, bool on) {
        const uint8_t *p = reinterpret_cast<const uint8_t *>(row) + at;
        uint32_t u[V * kSize / 4] = {};
        if (on) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if constexpr (FP32) u[j] = reinterpret_cast<const uint32_t *>(p)[j];
                else u[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(p)[j] << (j % 2 * 16);
            }
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            w[i] = uint4{u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]};
    }
    __device__ __forceinline__ void values(float (&f)[V]) const {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (FP32) f[4 * i + j] = __uint_as_float(u[j]);
                else f[2 * j] = bf16_lo(u[j]), f[2 * j + 1] = bf16_hi(u[j]);
            }
        }
    }
    __device__ __forceinline__ void set(const float (&f)[V]) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            if constexpr (FP32)
                w[i] = __builtin_bit_cast(uint4, float4{f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]});
            else
                w[i] = uint4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                             pack_bf16(f[6], f[7])};
        }
    }
    __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t at) const {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) bstore16(r, (int)(at + 16 * i), w[i]);
    }
    __device__ __forceinline__ void store_some(void *row, int at, bool on) const {
        if (!on) return;
        uint8_t *p = reinterpret_cast<uint8_t *>(row) + at;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint4 q = w[j * kSize / 16];
            const uint32_t u[4] = {q.x, q.y, q.z, q.w};
            if constexpr (FP32) reinterpret_cast<uint32_t *>(p)[j] = u[j % 4];
            else reinterpret_cast<uint16_t *>(p)[j] = (uint16_t)(u[j / 2 % 4] >> (j % 2 * 16));
        }
    }
};

// The heads of one token, rows of [heads][D]: piece i holds heads i kHeads, ...
template <bool FP32, int V, int LPV>
struct Heads {
    const uint8_t *row;
    __amdgpu_buffer_rsrc_t r;
    int heads;

    static constexpr int kHeads = kWave / LPV;
    __device__ __forceinline__ Heads(const void *x, int64_t at, int heads, int D)
        : row(reinterpret_cast<const uint8_t *>(x) + at * Raw<FP32, V>::kSize),
          r(make_rsrc(row, (int64_t)heads * D * Raw<FP32, V>::kSize)), heads(heads) {}
    static __device__ __forceinline__ int pieces(int heads) { return (heads + kHeads - 1) / kHeads; }
};

// LPV lanes a head, V values a lane; `parts` waves a token.
template <bool FP32, int MODE, int V, int LPV>
__global__ __launch_bounds__(256) void k_rope(RopeArgs a, int parts) {
    using Row = Heads<FP32, V, LPV>;
    using Values = Raw<FP32, V>;
    __shared__ RopeLds lds[4];
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int lane = threadIdx.x % kWave, d = lane % LPV * V, first = lane / LPV * LPV;
    const uint32_t unit = blockIdx.x * 4 + wave;
    const int64_t row = unit / (uint32_t)parts;
    if (row >= a.T) return;
    const int per = Row::pieces(a.heads), step = (per + parts - 1) / parts;
    const int i0 = (int)(unit % (uint32_t)parts) * step, i1 = min(i0 + step, per);
    const Row from(a.x, row * a.ldx, a.heads, a.D), to(a.out, row * a.ldo, a.heads, a.D);
    const uint32_t at = d < a.D ? (lane / LPV * a.D + d) * Values::kSize : kOOB;
    const uint32_t next = Row::kHeads * a.D * Values::kSize;
    auto on = [&](int i) { return d < a.D && i * Row::kHeads + lane / LPV < a.heads; };
    Values x[kAhead];
    auto load = [&](int i) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (i + u >= i1) break;
            if constexpr (MODE != kSome) x[u].template load<MODE>(from.r, at + (i + u) * next);
            else x[u].load_some(from.row, (int)(at + (i + u) * next), on(i + u));
        }
    };
    load(i0);  // (in flight while the angles are computed)
    const Turn<V> t = rope_turn<V>(a.rope, a.pos[row], d, lds[wave]);
    for (int i = i0; i < i1; i += kAhead) {
        if (i > i0) load(i);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (i + u >= i1) break;
            float f[V];
            x[u].values(f);
            rotate<V>(a.rope, t, first, lds[wave].swap, f);
            Values y;
            y.set(f);
            if constexpr (MODE != kSome) y.store(to.r, at + (i + u) * next);
            else y.store_some(const_cast<uint8_t *>(to.row), (int)(at + (i + u) * next), on(i + u));
        }
    }
}

// A token of the call: its position (-1: of no sequence, or skipped) and its
// place in head 0 of its page (-1: it has no page).
struct TokenPlace {
    int64_t pos, at;
};

__device__ __forceinline__ TokenPlace token_place(const KvView &c, const KvRows &r, int64_t row) {
    int64_t b = row, pos = 0;
    if (r.cu) {
        b = find_sequence(r.cu, r.B, row);
        if (row < r.cu[b] || row >= r.cu[b + 1]) return {-1, -1};
        pos = row - r.cu[b];
    }
    const int start = r.start[b];
    if (start < 0) return {-1, -1};
    pos += start;
    const int page = kv_page(c, c.table + b * c.W, pos);
    return {pos, page < 0 ? -1
                          : (((int64_t)page * c.heads) << c.shift) + (pos & ((1 << c.shift) - 1))};
}

// The pieces of a token are those of its queries, then of its keys, then of its
// values, each kind a whole number of pieces.
template <bool INT8, bool FP32, int MODE, int V, int LPV>
__global__ __launch_bounds__(256) void k_kv_append_rope(AppendRopeArgs a, int parts) {
    using Row = Heads<FP32, V, LPV>;
    using Values = Raw<FP32, V>;
    __shared__ RopeLds lds[4];
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int lane = threadIdx.x % kWave, d = lane % LPV * V, first = lane / LPV * LPV;
    const uint32_t unit = blockIdx.x * 4 + wave;
    const int64_t row = unit / (uint32_t)parts;
    if (row >= a.rows.T) return;
    const int D = a.c.D, heads = a.c.heads;
    const int nq = Row::pieces(a.hq), nk = Row::pieces(heads);
    const int per = nq + 2 * nk, step = (per + parts - 1) / parts;
    const int i0 = (int)(unit % (uint32_t)parts) * step, i1 = min(i0 + step, per);
    const Row q(a.q, row * a.ldq, a.hq, D), k(a.k, row * a.ldk, heads, D), v(a.v, row * a.ldv, heads, D);
    const Row to(a.out, row * a.ldo, a.hq, D);
    const uint32_t at = d < D ? (lane / LPV * D + d) * Values::kSize : kOOB;
    const uint32_t next = Row::kHeads * D * Values::kSize;
    Values x[kAhead];
    auto load = [&](int i) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int n = i + u;
            if (n >= i1) break;
            const int m = n < nq ? n : n < nq + nk ? n - nq : n - nq - nk;
            if constexpr (MODE != kSome) {
                x[u].template load<MODE>(n < nq ? q.r : n < nq + nk ? k.r : v.r, at + m * next);
            } else {
                x[u].load_some(n < nq ? q.row : n < nq + nk ? k.row : v.row, (int)(at + m * next),
                               d < D && m * Row::kHeads + lane / LPV < (n < nq ? a.hq : heads));
            }
        }
    };
    load(i0);  // (in flight during the search for the place, and while the angles are computed)
    const TokenPlace place = token_place(a.c, a.rows, row);
    if (place.pos < 0) return;
    const Turn<V> t = rope_turn<V>(a.rope, place.pos, d, lds[wave]);
    for (int i = i0; i < i1; i += kAhead) {
        if (i > i0) load(i);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int n = i + u;
            if (n >= i1) break;
            float f[V];
            x[u].values(f);
            if (n < nq + nk) rotate<V>(a.rope, t, first, lds[wave].swap, f);
            if (n < nq) {
                Values y;
                y.set(f);
                if constexpr (MODE != kSome) y.store(to.r, at + n * next);
                else y.store_some(const_cast<uint8_t *>(to.row), (int)(at + n * next),
                                  d < D && n * Row::kHeads + lane / LPV < a.hq);
            } else if (place.at >= 0) {
                const bool isv = n >= nq + nk;
                const int h = (isv ? n - nq - nk : n - nq) * Row::kHeads + lane / LPV;
                kv_store<INT8, V, LPV>(a.c, isv, place.at + ((int64_t)h << a.c.shift), d,
                                       h < heads && d < D, f);
            }
        }
    }
}

static bool aligned16(const void *p, int64_t stride, bool fp32) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride * (fp32 ? 4 : 2) % 16 == 0;
}

// Waves of a token: as many as its pieces, or 2048 of the call.
static int parts_of(int64_t T, int pieces) {
    return (int)std::max<int64_t>(1, std::min<int64_t>(pieces, 2048 / T));
}

// f(values of a lane, lanes of a head) for heads of D values: 16 bytes a lane, so
// that neighbouring lanes read side by side, while a head fits a wave.
template <bool FP32, typename F>
static void by_head(int D, F f) {
    constexpr int V = FP32 ? 4 : 8;
    if (D <= 8 * V) f(Int<V>{}, Int<8>{});
    else if (D <= 16 * V) f(Int<V>{}, Int<16>{});
    else if (D <= 32 * V) f(Int<V>{}, Int<32>{});
    else if (D <= 64 * V) f(Int<V>{}, Int<64>{});
    else f(Int<8>{}, Int<64>{});
}

template <bool FP32>
static void go_rope(const RopeArgs &a, const char **path, hipStream_t st) {
    const bool vec = aligned16(a.x, a.ldx, FP32) && aligned16(a.out, a.ldo, FP32);
    const bool lines = a.D * (FP32 ? 4 : 2) % 128 == 0;
    *path = !vec ? "rope_rotate_odd" : !lines ? "rope_rotate_cached" : "rope_rotate";
    by_head<FP32>(a.D, [&](auto v, auto lanes) {
        constexpr int V = decltype(v)::value, LPV = decltype(lanes)::value;
        const int parts = parts_of(a.T, (a.heads + kWave / LPV - 1) / (kWave / LPV));
        const dim3 g((unsigned)((a.T * parts + 3) / 4));
        if (!vec) launch_kv(k_rope<FP32, kSome, V, LPV>, g, dim3(256), 0, st, a, parts);
        else if (!lines) launch_kv(k_rope<FP32, kCached, V, LPV>, g, dim3(256), 0, st, a, parts);
        else launch_kv(k_rope<FP32, kStream, V, LPV>, g, dim3(256), 0, st, a, parts);
    });
}

hipError_t launch_rope(const RopeArgs &a, const char **path, hipStream_t st) {
    if (a.fp32) go_rope<true>(a, path, st);
    else go_rope<false>(a, path, st);
    return hipGetLastError();
}

template <bool INT8, bool FP32>
static void go_append(const AppendRopeArgs &a, const char **path, hipStream_t st) {
    const bool vec = aligned16(a.q, a.ldq, FP32) && aligned16(a.out, a.ldo, FP32) &&
                     aligned16(a.k, a.ldk, FP32) && aligned16(a.v, a.ldv, FP32);
    const bool lines = a.c.D * (FP32 ? 4 : 2) % 128 == 0;
    *path = !vec ? "kv_append_rope_odd" : !lines ? "kv_append_rope_cached" : "kv_append_rope";
    by_head<FP32>(a.c.D, [&](auto v, auto lanes) {
        constexpr int V = decltype(v)::value, LPV = decltype(lanes)::value, H = kWave / LPV;
        const int parts = parts_of(a.rows.T, (a.hq + H - 1) / H + 2 * ((a.c.heads + H - 1) / H));
        const dim3 g((unsigned)((a.rows.T * parts + 3) / 4));
        if (!vec) launch_kv(k_kv_append_rope<INT8, FP32, kSome, V, LPV>, g, dim3(256), 0, st, a, parts);
        else if (!lines) launch_kv(k_kv_append_rope<INT8, FP32, kCached, V, LPV>, g, dim3(256), 0, st, a, parts);
        else launch_kv(k_kv_append_rope<INT8, FP32, kStream, V, LPV>, g, dim3(256), 0, st, a, parts);
    });
}

hipError_t launch_kv_append_rope(const AppendRopeArgs &a, const char **path, hipStream_t st) {
    if (a.int8) a.fp32 ? go_append<true, true>(a, path, st) : go_append<true, false>(a, path, st);
    else a.fp32 ? go_append<false, true>(a, path, st) : go_append<false, false>(a, path, st);
    return hipGetLastError();
}

}  // namespace w4
