// Rotary norm of queries and keys (include/qkr.h), and the paged append
// (include/paged.h), which is the same pass with a cache for its output.
//
// One pass over the data: a vector of up to 128 channels lies in the registers
// of a few neighbouring lanes (da::QkrSide), its mean square is a sum over
// those lanes, and it is written back in the order in which it was read. The
// cosines and sines of a token are formed once, by the lanes of the warp that
// takes the token, and read by all of the token's heads from shared memory.
// The angle is a product modulo 2^64 of a 32-bit position and a 64-bit fraction
// of a turn; it is exact, so no position costs digits, and needs no 64-bit
// floating point.
//
// Measured, a call among others: 8,192 tokens of 8 heads (4 key heads) of 2 x 64
// in bf16, twice, forward and backward 75 us for 251 MB: 3.4 TB/s, half of what a
// copy reaches. The forward kernel issues on 60 % of its clocks and waits for
// loads on most others, the backward kernel the same: instructions and the
// latency of a warp's two vectors under way bound them together, not memory (25
// and 35 % busy). 4,095 tokens of 16 heads in fp16, forward: 14 us for 42 MB; a
// prompt's append, 4 x 4,095 tokens of 8 heads with values: 37 us for 134 MB. One
// token: 7 us, launch and latency. The forward forms with 16-byte pieces do not fit
// in the 80 registers that three CTAs to an SM leave: 200 B of a thread's are stored
// and 288 B read in bf16, 304 and 448 with a paged side. With two CTAs to an SM
// nothing is spilled and fewer warps hide the loads: 73 us for the first of these
// cases, but 16.4 for the second and 41 for the third. Four vectors under way, or
// one, with two to four CTAs to an SM: 77 to 110 us for the first, 17 to 23 for the
// second.
#include <cmath>
#include <cuda_bf16.h>

#include "qkr_internal.cuh"

namespace da {
namespace {

constexpr int kQkrThreads = 256;
constexpr int kQkrWarps = kQkrThreads / 32;
constexpr int kPairs = 128;  // cosines and sines that a warp holds
constexpr int kTokens = 32;  // tokens that a warp takes at most at once

template <int BYTES> struct QkrRaw;
template <> struct QkrRaw<16> { using type = uint4; };
template <> struct QkrRaw<8> { using type = uint2; };
template <> struct QkrRaw<4> { using type = uint32_t; };
template <> struct QkrRaw<2> { using type = unsigned short; };

// V channels as they lie in memory, and as pairs of floats (with one channel
// the second of the pair is zero). Arithmetic on pairs takes half the
// instructions, which bound these passes before memory does otherwise.
template <typename T, int V> using Piece = typename QkrRaw<static_cast<int>(sizeof(T)) * V>::type;
template <int V> constexpr int kPairsOf = (V + 1) / 2;

__device__ __forceinline__ float2 widen(uint32_t w, const __nv_bfloat16 *) { return {__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)}; }
__device__ __forceinline__ float2 widen(uint32_t w, const __half *) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }
__device__ __forceinline__ uint32_t narrow(float2 v, const __nv_bfloat16 *)
{
    const __nv_bfloat162 r = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t narrow(float2 v, const __half *)
{
    const __half2 r = __floats2half2_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t *>(&r);
}

template <typename T, int V> __device__ __forceinline__ void unpack(const Piece<T, V> &p, float2 (&f)[kPairsOf<V>])
{
    if constexpr (sizeof(T) == 4) {
        const float *x = reinterpret_cast<const float *>(&p);
#pragma unroll
        for (int i = 0; i < kPairsOf<V>; ++i) f[i] = {x[2 * i], V == 1 ? 0.f : x[2 * i + (V > 1)]};
    } else if constexpr (V == 1) {
        f[0] = {widen(p, static_cast<const T *>(nullptr)).x, 0.f};
    } else {
        const uint32_t *x = reinterpret_cast<const uint32_t *>(&p);
#pragma unroll
        for (int i = 0; i < kPairsOf<V>; ++i) f[i] = widen(x[i], static_cast<const T *>(nullptr));
    }
}

template <typename T, int V> __device__ __forceinline__ Piece<T, V> pack(const float2 (&f)[kPairsOf<V>])
{
    Piece<T, V> p;
    if constexpr (sizeof(T) == 4) {
        float *x = reinterpret_cast<float *>(&p);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = i % 2 ? f[i / 2].y : f[i / 2].x;
    } else if constexpr (V == 1) {
        p = static_cast<unsigned short>(narrow(f[0], static_cast<const T *>(nullptr)) & 0xffffu);
    } else {
        uint32_t *x = reinterpret_cast<uint32_t *>(&p);
#pragma unroll
        for (int i = 0; i < kPairsOf<V>; ++i) x[i] = narrow(f[i], static_cast<const T *>(nullptr));
    }
    return p;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)), "l"(reinterpret_cast<uint64_t &>(c)));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}
__device__ __forceinline__ float2 minus(float2 a) { return {-a.x, -a.y}; }

// A lane's two pieces of each of its slots: SPL slots, 2 V channels each.
template <int V> constexpr int kSlots = V >= 4 ? 1 : V == 2 ? 2 : 4;

struct Slot {
    int a, b;      // first channels of the pieces, or -1
    int pair;      // first pair, or -1
};

template <int V> __device__ __forceinline__ Slot slot_of(const QkrSide &s, int t, int interleaved)
{
    Slot r{-1, -1, -1};
    if (t < s.nr) {
        r.a = interleaved ? t * 2 * V : t * V;
        r.b = interleaved ? r.a + V : s.R / 2 + r.a;
        r.pair = t * V;
    } else if (t < s.slots) {
        r.a = s.R + (t - s.nr) * 2 * V;
        r.b = r.a + V < s.D ? r.a + V : -1;
    }
    return r;
}

template <int V> __device__ __forceinline__ void weights_of(const QkrSide &s, int at, float2 (&w)[kPairsOf<V>])
{
#pragma unroll
    for (int i = 0; i < kPairsOf<V>; ++i)
        w[i] = {s.w && at >= 0 ? s.w[at + 2 * i] : 1.f, V > 1 && s.w && at >= 0 ? s.w[at + 2 * i + 1] : 1.f};
}

// Cosine and sine of pos * turns / 2^64 of a turn: the product's quarter turn
// next to it exactly, the rest, an angle of at most pi / 4, to 2^-34 of a turn
// and then by the first terms of their Taylor series, whose next ones are below
// 2^-25 there.
__device__ __forceinline__ float2 angle(int pos, int64_t turns)
{
    const uint64_t at = static_cast<uint64_t>(static_cast<int64_t>(pos)) * static_cast<uint64_t>(turns);
    const uint32_t quarter = static_cast<uint32_t>((at + (uint64_t{1} << 61)) >> 62);
    const int64_t rest = static_cast<int64_t>(at - (static_cast<uint64_t>(quarter) << 62));
    const float x = static_cast<float>(static_cast<int32_t>(rest >> 30)) * 3.657295198e-10f, y = x * x;  // 2 pi / 2^34
    const float s = fmaf(x * y, fmaf(y, fmaf(y, fmaf(y, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), x);
    const float c = fmaf(y, fmaf(y, fmaf(y, fmaf(y, fmaf(y, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -0.5f), 1.f);
    const float u = quarter & 1 ? -s : c, v = quarter & 1 ? c : s;
    return (quarter & 2) ? make_float2(-u, -v) : make_float2(u, v);
}

// What a warp has in shared memory: its tokens' angles, and where they lie.
struct WarpTokens {
    float c[kPairs], s[kPairs];       // [token][R / 2], times the magnitude
    int64_t from[kTokens], to[kTokens];  // first element of a token's vectors, or to < 0: not to be stored
};

// Which tokens a warp's vectors are of.
struct Run {
    int64_t token0;
    int count;     // tokens
};

// Where a run's tokens lie; paged: by page and place.
template <bool PAGED> __device__ __forceinline__ void fill_places(const QkrArgs &a, const QkrSide &s, const Run &run, WarpTokens &w)
{
    for (int t = threadIdx.x & 31; t < run.count; t += 32) {
        const int64_t token = run.token0 + t;
        const int b = static_cast<int>(s.div_L.div(static_cast<uint32_t>(token))), l = static_cast<int>(token - static_cast<int64_t>(b) * s.L);
        w.from[t] = b * s.xs[0] + l * s.xs[1];
        int64_t to = b * s.ys[0] + l * s.ys[1];
        if (PAGED && s.paged) {
            to = -1;
            const int64_t place = static_cast<int64_t>(a.lengths[b]) + l;
            if (l < (a.counts ? a.counts[b] : s.L) && place >= 0 && place < static_cast<int64_t>(a.table_pages) * a.page_size) {
                const int n = static_cast<int>(a.div_page.div(static_cast<uint32_t>(place)));
                const int page = a.table[static_cast<int64_t>(b) * a.table_pages + n];
                if (page >= 0 && page < a.num_pages) to = page * s.ys[0] + (place - static_cast<int64_t>(n) * a.page_size) * s.ys[1];
            }
        }
        w.to[t] = to;
    }
}

// The angles of a run's tokens.
__device__ __forceinline__ void fill_angles(const QkrArgs &a, const QkrSide &s, const Run &run, WarpTokens &w)
{
    const int hp = s.R / 2;
    for (int i = threadIdx.x & 31; i < run.count * hp; i += 32) {
        const int t = run.count == 1 ? 0 : static_cast<int>(s.div_hp.div(i));
        const int64_t token = run.token0 + t;
        int pos;
        if (s.pos) {
            pos = s.pos[token];
        } else {
            const int b = static_cast<int>(s.div_L.div(static_cast<uint32_t>(token)));
            const uint32_t l = static_cast<uint32_t>(token - static_cast<int64_t>(b) * s.L);
            pos = static_cast<int>(static_cast<uint32_t>(a.lengths ? a.lengths[b] : s.first) + l);
        }
        const float2 v = angle(pos, a.turns[i - t * hp]);
        w.c[i] = v.x * a.magnitude;
        w.s[i] = v.y * a.magnitude;
    }
}

// V angles' cosines or sines as pairs; they lie on multiples of V.
template <int V> __device__ __forceinline__ void load_angles(const float *p, float2 (&v)[kPairsOf<V>])
{
    if constexpr (V >= 4) {
#pragma unroll
        for (int j = 0; j < V / 4; ++j) {
            const float4 x = reinterpret_cast<const float4 *>(p)[j];
            v[2 * j] = {x.x, x.y};
            v[2 * j + 1] = {x.z, x.w};
        }
    } else if constexpr (V == 2) {
        v[0] = *reinterpret_cast<const float2 *>(p);
    } else {
        v[0] = {*p, 0.f};
    }
}

// z_a, z_b of the pairs of a slot; BACK: the turn in the other direction.
template <int V, bool BACK>
__device__ __forceinline__ void turn(const float *c, const float *s, int interleaved, float2 (&a)[kPairsOf<V>], float2 (&b)[kPairsOf<V>])
{
    constexpr int P = kPairsOf<V>;
    float2 u[P], v[P];
    load_angles<V>(c, u);
    load_angles<V>(s, v);
    if (V > 1 && interleaved) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            // Pair j of piece a turns by angle j, of piece b by angle V / 2 + j.
            constexpr int half = V / 2;
            const float c0 = j % 2 ? u[j / 2].y : u[j / 2].x, s0 = BACK ? -(j % 2 ? v[j / 2].y : v[j / 2].x) : j % 2 ? v[j / 2].y : v[j / 2].x;
            const int k = half + j;
            const float c1 = k % 2 ? u[k / 2].y : u[k / 2].x, s1 = BACK ? -(k % 2 ? v[k / 2].y : v[k / 2].x) : k % 2 ? v[k / 2].y : v[k / 2].x;
            const float2 x = a[j], y = b[j];
            a[j] = {x.x * c0 - x.y * s0, x.x * s0 + x.y * c0};
            b[j] = {y.x * c1 - y.y * s1, y.x * s1 + y.y * c1};
        }
    } else {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const float2 x = a[j], y = b[j], n = minus(v[j]);
            a[j] = fma2(y, BACK ? v[j] : n, mul2(x, u[j]));
            b[j] = fma2(x, BACK ? n : v[j], mul2(y, u[j]));
        }
    }
}

__device__ __forceinline__ float lanes_sum(float v, int sg_log2)
{
    for (int o = 1 << sg_log2 >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A piece, zeros where there is none.
template <typename T, int V> __device__ __forceinline__ Piece<T, V> load_piece(const T *base, int at, bool live)
{
    Piece<T, V> p{};
    if (live && at >= 0) p = __ldcs(reinterpret_cast<const Piece<T, V> *>(base + at));
    return p;
}
template <typename T, int V> __device__ __forceinline__ void store_piece(T *base, int at, const float2 (&f)[kPairsOf<V>])
{
    if (at >= 0) *reinterpret_cast<Piece<T, V> *>(base + at) = pack<T, V>(f);
}

// Vectors that a group of lanes has under way at once.
constexpr int kAhead = 2;

// ---- forward, and append ---------------------------------------------------

template <typename T, int V, bool PAGED>
__device__ __forceinline__ void forward_side(const QkrArgs &a, const QkrSide &s, WarpTokens &w)
{
    constexpr int SPL = kSlots<V>, P = kPairsOf<V>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lanes = 1 << s.sg_log2, sub = lane >> s.sg_log2, step = 32 >> s.sg_log2, HM = s.H * s.M;
    Slot slot[SPL];
    float2 wa[SPL][P], wb[SPL][P];
#pragma unroll
    for (int p = 0; p < SPL; ++p) {
        slot[p] = slot_of<V>(s, (lane & (lanes - 1)) + p * 32, a.interleaved);
        weights_of<V>(s, slot[p].a, wa[p]);
        weights_of<V>(s, slot[p].b, wb[p]);
    }
    // A warp's turns: runs of tokens, or parts of one token's vectors.
    for (int64_t of = (blockIdx.x - s.unit0) * kQkrWarps + warp;; of += static_cast<int64_t>(s.units) * kQkrWarps) {
    const int64_t part = s.parts > 1 ? of % s.parts : 0;
    Run run;
    run.token0 = s.parts > 1 ? of / s.parts : of * s.tpw;
    if (run.token0 >= s.tokens) return;
    run.count = static_cast<int>(min(static_cast<int64_t>(s.tpw), s.tokens - run.token0));
    __syncwarp();  // the turn before has been read
    fill_places<PAGED>(a, s, run, w);
    __syncwarp();
    const int begin = static_cast<int>(part) * s.per, vectors = s.parts > 1 ? min(begin + s.per, HM) : run.count * HM;
    Piece<T, V> xa[kAhead][SPL], xb[kAhead][SPL];
    int at[kAhead];  // the vector's token and place in it, or -1
    const auto fetch = [&](int i0) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u * step;
            const bool live = i < vectors;
            const int t = live ? static_cast<int>(s.div_vec.div(i)) : 0, hm = i - t * HM, h = s.M == 2 ? hm >> 1 : hm, m = s.M == 2 ? hm & 1 : 0;
            const T *x = static_cast<const T *>(s.x) + w.from[t] + h * s.xs[2] + m * s.xs[3];
#pragma unroll
            for (int p = 0; p < SPL; ++p) {
                xa[u][p] = load_piece<T, V>(x, slot[p].a, live);
                xb[u][p] = load_piece<T, V>(x, slot[p].b, live);
            }
            at[u] = live ? i : -1;
        }
    };
    fetch(begin + sub);
    fill_angles(a, s, run, w);
    __syncwarp();

    for (int i0 = begin + sub; i0 - sub < vectors; i0 += kAhead * step) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = at[u], t = i >= 0 ? static_cast<int>(s.div_vec.div(i)) : 0;
            float2 fa[SPL][P], fb[SPL][P], sq = {0.f, 0.f};
#pragma unroll
            for (int p = 0; p < SPL; ++p) {
                unpack<T, V>(xa[u][p], fa[p]);
                unpack<T, V>(xb[u][p], fb[p]);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    sq = fma2(fa[p][j], fa[p][j], sq);
                    sq = fma2(fb[p][j], fb[p][j], sq);
                }
            }
            if (s.normed) {
                const float r1 = rsqrtf(fmaf(lanes_sum(sq.x + sq.y, s.sg_log2), s.inv_D, a.eps));
                const float2 r = {r1, r1};
#pragma unroll
                for (int p = 0; p < SPL; ++p)
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        fa[p][j] = mul2(mul2(fa[p][j], r), wa[p][j]);
                        fb[p][j] = mul2(mul2(fb[p][j], r), wb[p][j]);
                    }
            }
            const int64_t to = w.to[t];
            if (i < 0 || (PAGED && to < 0)) continue;
            const int hm = i - t * HM, h = s.M == 2 ? hm >> 1 : hm, m = s.M == 2 ? hm & 1 : 0;
            T *y = static_cast<T *>(s.y) + to + h * s.ys[2] + m * s.ys[3];
#pragma unroll
            for (int p = 0; p < SPL; ++p) {
                if (slot[p].pair >= 0) {
                    const int k = t * (s.R / 2) + slot[p].pair;
                    turn<V, false>(w.c + k, w.s + k, a.interleaved, fa[p], fb[p]);
                }
                store_piece<T, V>(y, slot[p].a, fa[p]);
                store_piece<T, V>(y, slot[p].b, fb[p]);
            }
        }
        if (i0 - sub + kAhead * step < vectors) fetch(i0 + kAhead * step);
    }
    }
}

// A CTA's side. The sides are told apart here and not by an index, so that their
// fields are operands of instructions and not loads.
__device__ __forceinline__ int which_side(const QkrArgs &a)
{
    const int64_t cta = blockIdx.x;
    return a.sides > 2 && cta >= a.side[2].unit0 ? 2 : a.sides > 1 && cta >= a.side[1].unit0 ? 1 : 0;
}

template <typename T, int V, bool PAGED>
__global__ void __launch_bounds__(kQkrThreads, 3) qkr_forward_kernel(const __grid_constant__ QkrArgs a)
{
    __shared__ __align__(16) WarpTokens all[kQkrWarps];
    WarpTokens &w = all[threadIdx.x >> 5];
    const int which = which_side(a);
    if (which == 0) forward_side<T, V, PAGED>(a, a.side[0], w);
    else if (which == 1) forward_side<T, V, PAGED>(a, a.side[1], w);
    else if (PAGED) forward_side<T, V, PAGED>(a, a.side[2], w);
}

// ---- backward --------------------------------------------------------------

// CTAs of a side walk over its runs; every lane sums its channels' part of the
// weight's gradient over all of its vectors in registers, and a CTA leaves one
// row of sums.
template <typename T, int V>
__device__ __forceinline__ void backward_side(const QkrArgs &a, const QkrSide &s, WarpTokens &w, float (&sums)[kQkrWarps][QKR_MAX_WIDTH])
{
    constexpr int SPL = kSlots<V>, P = kPairsOf<V>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = static_cast<int>(blockIdx.x - s.unit0);
    const int lanes = 1 << s.sg_log2, sub = lane >> s.sg_log2, step = 32 >> s.sg_log2, HM = s.H * s.M;
    Slot slot[SPL];
    float2 wa[SPL][P], wb[SPL][P], ga[SPL][P], gb[SPL][P];
#pragma unroll
    for (int p = 0; p < SPL; ++p) {
        slot[p] = slot_of<V>(s, (lane & (lanes - 1)) + p * 32, a.interleaved);
        weights_of<V>(s, slot[p].a, wa[p]);
        weights_of<V>(s, slot[p].b, wb[p]);
#pragma unroll
        for (int j = 0; j < P; ++j) ga[p][j] = gb[p][j] = {0.f, 0.f};
    }
    for (int64_t r = static_cast<int64_t>(cta) * kQkrWarps + warp; r * s.tpw < s.tokens; r += static_cast<int64_t>(s.units) * kQkrWarps) {
        Run run;
        run.token0 = r * s.tpw;
        run.count = static_cast<int>(min(static_cast<int64_t>(s.tpw), s.tokens - run.token0));
        const int vectors = run.count * HM;
        __syncwarp();  // the run before has been read
        fill_places<false>(a, s, run, w);
        __syncwarp();
        Piece<T, V> xa[kAhead][SPL], xb[kAhead][SPL], za[kAhead][SPL], zb[kAhead][SPL];
        const auto fetch = [&](int i0) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = i0 + u * step;
                const bool live = i < vectors;
                const int t = live ? static_cast<int>(s.div_vec.div(i)) : 0, hm = i - t * HM;
                const T *x = static_cast<const T *>(s.x) + w.from[t] + (hm >> 1) * s.xs[2] + (hm & 1) * s.xs[3];
                const T *g = static_cast<const T *>(s.g) + (run.token0 * HM + i) * s.D;
#pragma unroll
                for (int p = 0; p < SPL; ++p) {
                    za[u][p] = load_piece<T, V>(g, slot[p].a, live);
                    zb[u][p] = load_piece<T, V>(g, slot[p].b, live);
                    xa[u][p] = load_piece<T, V>(x, slot[p].a, live && s.normed);
                    xb[u][p] = load_piece<T, V>(x, slot[p].b, live && s.normed);
                }
            }
        };
        fetch(sub);
        fill_angles(a, s, run, w);
        __syncwarp();
        for (int i0 = sub; i0 - sub < vectors; i0 += kAhead * step) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = i0 + u * step;
                const bool live = i < vectors;
                const int t = live ? static_cast<int>(s.div_vec.div(i)) : 0;
                float2 ha[SPL][P], hb[SPL][P];
#pragma unroll
                for (int p = 0; p < SPL; ++p) {
                    unpack<T, V>(za[u][p], ha[p]);
                    unpack<T, V>(zb[u][p], hb[p]);
                    if (slot[p].pair >= 0) {
                        const int k = t * (s.R / 2) + slot[p].pair;
                        turn<V, true>(w.c + k, w.s + k, a.interleaved, ha[p], hb[p]);
                    }
                }
                if (s.normed) {
                    float2 na[SPL][P], nb[SPL][P], sq = {0.f, 0.f}, dot = {0.f, 0.f};
#pragma unroll
                    for (int p = 0; p < SPL; ++p) {
                        unpack<T, V>(xa[u][p], na[p]);
                        unpack<T, V>(xb[u][p], nb[p]);
#pragma unroll
                        for (int j = 0; j < P; ++j) {
                            sq = fma2(na[p][j], na[p][j], sq);
                            sq = fma2(nb[p][j], nb[p][j], sq);
                        }
                    }
                    const float rn = rsqrtf(fmaf(lanes_sum(sq.x + sq.y, s.sg_log2), s.inv_D, a.eps));
                    const float2 r2 = {rn, rn};
#pragma unroll
                    for (int p = 0; p < SPL; ++p)
#pragma unroll
                        for (int j = 0; j < P; ++j) {
                            na[p][j] = mul2(na[p][j], r2);
                            nb[p][j] = mul2(nb[p][j], r2);
                            ga[p][j] = fma2(ha[p][j], na[p][j], ga[p][j]);
                            gb[p][j] = fma2(hb[p][j], nb[p][j], gb[p][j]);
                            ha[p][j] = mul2(ha[p][j], wa[p][j]);
                            hb[p][j] = mul2(hb[p][j], wb[p][j]);
                            dot = fma2(ha[p][j], na[p][j], dot);
                            dot = fma2(hb[p][j], nb[p][j], dot);
                        }
                    const float mean = -lanes_sum(dot.x + dot.y, s.sg_log2) * s.inv_D;
                    const float2 m2 = {mean, mean};
#pragma unroll
                    for (int p = 0; p < SPL; ++p)
#pragma unroll
                        for (int j = 0; j < P; ++j) {
                            ha[p][j] = mul2(r2, fma2(na[p][j], m2, ha[p][j]));
                            hb[p][j] = mul2(r2, fma2(nb[p][j], m2, hb[p][j]));
                        }
                }
                if (!live) continue;
                T *y = static_cast<T *>(s.y) + (run.token0 * HM + i) * s.D;
#pragma unroll
                for (int p = 0; p < SPL; ++p) {
                    store_piece<T, V>(y, slot[p].a, ha[p]);
                    store_piece<T, V>(y, slot[p].b, hb[p]);
                }
            }
            if (i0 - sub + kAhead * step < vectors) fetch(i0 + kAhead * step);
        }
    }
    if (!s.part) return;
#pragma unroll
    for (int p = 0; p < SPL; ++p)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float x = j % 2 ? ga[p][j / 2].y : ga[p][j / 2].x, y = j % 2 ? gb[p][j / 2].y : gb[p][j / 2].x;
            for (int o = lanes; o < 32; o <<= 1) {
                x += __shfl_xor_sync(0xffffffffu, x, o);
                y += __shfl_xor_sync(0xffffffffu, y, o);
            }
            if (sub == 0) {
                if (slot[p].a >= 0) sums[warp][slot[p].a + j] = x;
                if (slot[p].b >= 0) sums[warp][slot[p].b + j] = y;
            }
        }
    __syncthreads();
    for (int d = threadIdx.x; d < s.D; d += kQkrThreads) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < kQkrWarps; ++k) t += sums[k][d];
        s.part[static_cast<int64_t>(cta) * s.D + d] = t;
    }
}

template <typename T, int V> __global__ void __launch_bounds__(kQkrThreads, 2) qkr_backward_kernel(const __grid_constant__ QkrArgs a)
{
    __shared__ __align__(16) WarpTokens all[kQkrWarps];
    __shared__ float sums[kQkrWarps][QKR_MAX_WIDTH];
    WarpTokens &w = all[threadIdx.x >> 5];
    if (which_side(a) == 0) backward_side<T, V>(a, a.side[0], w, sums);
    else backward_side<T, V>(a, a.side[1], w, sums);
}

// grad_weight of a side: the CTAs' rows in a fixed order. A block takes 32
// channels, its 32 warps share the rows.
__global__ void __launch_bounds__(1024) qkr_weight_kernel(const __grid_constant__ QkrArgs a)
{
    __shared__ float sums[32][33];
    const QkrSide &s = a.side[blockIdx.y];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = blockIdx.x * 32 + lane;
    pdl_wait();
    if (!s.part) return;
    float t = 0.f;
    if (d < s.D)
#pragma unroll 4
        for (int c = warp; c < s.units; c += 32) t += s.part[static_cast<int64_t>(c) * s.D + d];
    sums[warp][lane] = t;
    __syncthreads();
    t = lanes_sum(sums[lane][warp], 5);  // of channel blockIdx.x * 32 + warp
    if (lane == 0 && blockIdx.x * 32 + warp < s.D) s.grad_w[blockIdx.x * 32 + warp] = t;
}

// ---- host ------------------------------------------------------------------

bool piece_fits(const QkrSide &s, int elem, int V, bool backward)
{
    if (s.D % V || s.R / 2 % V) return false;
    if (!aligned(s.x, V * elem) || !aligned(s.y, V * elem) || (backward && !aligned(s.g, V * elem))) return false;
    const int64_t n[4] = {s.tokens / s.L, s.L, s.H, s.M};
    for (int i = 0; i < 4; ++i)
        if (n[i] > 1 && (s.xs[i] % V || s.ys[i] % V)) return false;
    return s.ys[0] % V == 0 && (!s.paged || s.ys[1] % V == 0);
}

// Fills what depends on the width of a piece; returns that width.
int plan_sides(QkrArgs &a, int elem, bool backward)
{
    int V = 16 / elem;
    for (int i = 0; i < a.sides; ++i)
        while (!piece_fits(a.side[i], elem, V, backward)) V /= 2;
    for (int i = 0; i < a.sides; ++i) {
        QkrSide &s = a.side[i];
        s.nr = s.R / 2 / V;
        s.slots = s.nr + ((s.D - s.R) / V + 1) / 2;
        s.sg_log2 = 0;
        while ((1 << s.sg_log2) < s.slots && s.sg_log2 < 5) ++s.sg_log2;
        // Enough tokens to give every group of lanes two vectors at a time,
        // unless that leaves SMs without warps.
        const int vec = s.H * s.M, want = kAhead * (32 >> s.sg_log2);
        int tpw = (want + vec - 1) / vec;
        while (tpw > 1 && (s.tokens / tpw < 152 * 16 || tpw * (s.R / 2) > kPairs || tpw > kTokens)) tpw = (tpw + 1) / 2;
        s.tpw = tpw;
        // Few tokens of many heads: warps share a token, two vectors at a time each.
        s.parts = 1;
        s.per = vec;
        if (!backward && tpw == 1 && vec > want)
            while (s.parts < 16 && s.tokens * s.parts < 152 * 8 && vec > want * s.parts) s.parts *= 2;
        if (s.parts > 1) {
            s.per = ((vec + s.parts - 1) / s.parts + 1) / 2 * 2;
            s.parts = (vec + s.per - 1) / s.per;
        }
        s.div_L = FastDiv::make(static_cast<uint32_t>(s.L));
        s.div_vec = FastDiv::make(static_cast<uint32_t>(vec));
        s.div_hp = FastDiv::make(static_cast<uint32_t>(s.R > 0 ? s.R / 2 : 1));
    }
    return V;
}

template <typename T, int V> cudaError_t forward_paged(const QkrArgs &a, unsigned grid, cudaStream_t st)
{
    if (a.table || a.lengths) qkr_forward_kernel<T, V, true><<<grid, kQkrThreads, 0, st>>>(a);
    else qkr_forward_kernel<T, V, false><<<grid, kQkrThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T> cudaError_t forward_pieces(const QkrArgs &a, int V, unsigned grid, cudaStream_t st)
{
    if constexpr (sizeof(T) == 2)
        if (V == 8) return forward_paged<T, 8>(a, grid, st);
    return V == 4 ? forward_paged<T, 4>(a, grid, st) : V == 2 ? forward_paged<T, 2>(a, grid, st) : forward_paged<T, 1>(a, grid, st);
}

template <typename T, int V> cudaError_t backward_run(const QkrArgs &a, unsigned grid, cudaStream_t st)
{
    qkr_backward_kernel<T, V><<<grid, kQkrThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T> cudaError_t backward_pieces(const QkrArgs &a, int V, unsigned grid, cudaStream_t st)
{
    if constexpr (sizeof(T) == 2)
        if (V == 8) return backward_run<T, 8>(a, grid, st);
    return V == 4 ? backward_run<T, 4>(a, grid, st) : V == 2 ? backward_run<T, 2>(a, grid, st) : backward_run<T, 1>(a, grid, st);
}

// CTAs of all sides together where their warps take many turns, as many as are
// resident: a warp then sets up once.
constexpr int kBackwardCtas = 152 * 2, kForwardCtas = 152 * 3;

// CTAs of each side, in proportion to its vectors; in the forward pass a warp
// for each turn where it would take fewer than `least` of them, because turns
// that do not come out even leave SMs idle at the end.
unsigned share_ctas(QkrArgs &a, int ctas, int least)
{
    int64_t all = 0, unit = 0, every = 0;
    for (int i = 0; i < a.sides; ++i) {
        all += a.side[i].tokens * a.side[i].H;
        every += (a.side[i].tokens + a.side[i].tpw - 1) / a.side[i].tpw * a.side[i].parts;
    }
    const bool one = every < static_cast<int64_t>(ctas) * kQkrWarps * least;
    for (int i = 0; i < a.sides; ++i) {
        QkrSide &s = a.side[i];
        const int64_t turns = (s.tokens + s.tpw - 1) / s.tpw * s.parts, most = (turns + kQkrWarps - 1) / kQkrWarps;
        const int64_t n = static_cast<int64_t>(static_cast<double>(ctas) * s.tokens * s.H / all);
        s.units = static_cast<int32_t>(one ? most : n < 1 ? 1 : n < most ? n : most);
        s.unit0 = unit;
        unit += s.units;
    }
    return static_cast<unsigned>(unit);
}

size_t part_bytes(const QkrSide &s) { return (static_cast<size_t>(kBackwardCtas + 1) * s.D * sizeof(float) + 255) & ~size_t{255}; }

}  // namespace

da_status qkr_sides(const qkr_problem *pr, const void *out_q, const void *out_k, QkrArgs &a)
{
    if (!pr) return fail(DA_ERR_NULL, "problem is NULL");
    const qkr_problem &p = *pr;
    if (p.batch < 0 || p.num_queries < 0 || p.num_keys < 0) return fail(DA_ERR_SHAPE, "negative size");
    if (p.num_heads < 1 || p.num_kv_heads < 1) return fail(DA_ERR_SHAPE, "num_heads and num_kv_heads must be positive");
    if (p.width < 1) return fail(DA_ERR_SHAPE, "width %d must be positive", p.width);
    if (p.width > QKR_MAX_WIDTH) return fail(DA_ERR_UNSUPPORTED, "width %d exceeds %d", p.width, QKR_MAX_WIDTH);
    if (p.rotated < 0 || p.rotated > p.width || p.rotated % 2)
        return fail(DA_ERR_SHAPE, "rotated (%d) must be even and at most width (%d)", p.rotated, p.width);
    if (p.dtype != DA_F32 && p.dtype != DA_BF16 && p.dtype != DA_F16) return fail(DA_ERR_SHAPE, "unknown dtype %d", p.dtype);
    if (p.normed && !(p.eps > 0.f && std::isfinite(p.eps))) return fail(DA_ERR_SHAPE, "eps must be positive and finite");
    if (!p.normed && (p.q_weight || p.k_weight)) return fail(DA_ERR_SHAPE, "a weight needs the norm");
    if (!std::isfinite(p.magnitude)) return fail(DA_ERR_SHAPE, "magnitude must be finite");
    for (int i = 0; i < 4; ++i)
        if (p.q_stride[i] < 0 || p.k_stride[i] < 0) return fail(DA_ERR_SHAPE, "strides must not be negative");
    const int64_t most = INT32_MAX;
    if (static_cast<int64_t>(p.batch) * p.num_queries > most || static_cast<int64_t>(p.batch) * p.num_keys > most ||
        p.num_heads > (1 << 20) || p.num_kv_heads > (1 << 20))
        return fail(DA_ERR_UNSUPPORTED, "more than 2^31 - 1 tokens, or than 2^20 heads");
    const int elem = p.dtype == DA_F32 ? 4 : 2;
    const void *elems[] = {p.q, p.k, out_q, out_k}, *words[] = {p.q_weight, p.k_weight, p.pos_q, p.pos_k};
    for (const void *x : elems)
        if (!aligned(x, elem)) return fail(DA_ERR_ALIGN, "q, k, outputs and gradients must be aligned to their elements");
    for (const void *x : words)
        if (!aligned(x, 4)) return fail(DA_ERR_ALIGN, "fp32 and int32 tensors must be 4-byte aligned");
    if (!aligned(p.turns, 8)) return fail(DA_ERR_ALIGN, "turns must be 8-byte aligned");
    a.sides = 0;
    a.interleaved = p.interleaved != 0;
    a.turns = p.turns;
    a.eps = p.eps;
    a.magnitude = p.magnitude;
    for (int i = 0; i < 2; ++i) {
        const int64_t L = i ? p.num_keys : p.num_queries;
        if (p.batch * L == 0) continue;
        if (!(i ? p.k : p.q)) return fail(DA_ERR_NULL, "%s is NULL", i ? "k" : "q");
        if (p.rotated > 0 && !p.turns) return fail(DA_ERR_NULL, "turns is NULL");
        QkrSide &s = a.side[a.sides++];
        s = QkrSide{};
        s.x = i ? p.k : p.q;
        s.y = const_cast<void *>(i ? out_k : out_q);
        s.H = i ? p.num_kv_heads : p.num_heads;
        s.M = 2;
        s.D = p.width;
        s.keys = i;
        s.inv_D = 1.f / static_cast<float>(p.width);
        s.R = p.rotated;
        s.L = static_cast<int32_t>(L);
        for (int j = 0; j < 4; ++j) s.xs[j] = i ? p.k_stride[j] : p.q_stride[j];
        s.ys[3] = s.D;
        s.ys[2] = 2 * s.D;
        s.ys[1] = s.ys[2] * s.H;
        s.ys[0] = s.ys[1] * L;
        s.w = i ? p.k_weight : p.q_weight;
        s.pos = i ? p.pos_k : p.pos_q;
        s.first = i || p.num_keys == 0 ? 0 : p.num_keys - p.num_queries;
        s.normed = p.normed != 0;
        s.tokens = p.batch * L;
    }
    return DA_OK;
}

da_status qkr_launch_forward(QkrArgs &a, int dtype, cudaStream_t st)
{
    if (a.sides == 0) return DA_OK;
    const int V = plan_sides(a, dtype == DA_F32 ? 4 : 2, false);
    const unsigned grid = share_ctas(a, kForwardCtas, 4);
    const cudaError_t e = dtype == DA_F32    ? forward_pieces<float>(a, V, grid, st)
                          : dtype == DA_BF16 ? forward_pieces<__nv_bfloat16>(a, V, grid, st)
                                             : forward_pieces<__half>(a, V, grid, st);
    return e == cudaSuccess ? DA_OK : cuda_fail(e, "rotary norm launch");
}

}  // namespace da

extern "C" {

da_status qkr_forward(const qkr_problem *p, void *out_q, void *out_k, da_stream_t stream)
{
    da::QkrArgs a{};
    const da_status st = da::qkr_sides(p, out_q, out_k, a);
    if (st != DA_OK) return st;
    for (int i = 0; i < a.sides; ++i)
        if (!a.side[i].y) return da::fail(DA_ERR_NULL, "out_q or out_k is NULL");
    return da::qkr_launch_forward(a, p->dtype, reinterpret_cast<cudaStream_t>(stream));
}

da_status qkr_workspace_size(const qkr_problem *p, size_t *bytes)
{
    if (!bytes) return da::fail(DA_ERR_NULL, "bytes is NULL");
    da::QkrArgs a{};
    const da_status st = da::qkr_sides(p, nullptr, nullptr, a);
    if (st != DA_OK) return st;
    *bytes = 0;
    for (int i = 0; i < a.sides; ++i)
        if (a.side[i].w) *bytes += da::part_bytes(a.side[i]);
    return DA_OK;
}

da_status qkr_backward(const qkr_problem *p, const void *grad_out_q, const void *grad_out_k, void *grad_q, void *grad_k,
                       float *grad_q_weight, float *grad_k_weight, void *workspace, size_t workspace_bytes,
                       da_stream_t stream)
{
    da::QkrArgs a{};
    da_status st = da::qkr_sides(p, grad_q, grad_k, a);
    if (st != DA_OK) return st;
    const int elem = p->dtype == DA_F32 ? 4 : 2;
    if ((p->q_weight == nullptr) != (grad_q_weight == nullptr) || (p->k_weight == nullptr) != (grad_k_weight == nullptr))
        return da::fail(DA_ERR_NULL, "a weight and its gradient go together");
    if (!da::aligned(grad_q_weight, 4) || !da::aligned(grad_k_weight, 4) || !da::aligned(grad_out_q, elem) || !da::aligned(grad_out_k, elem))
        return da::fail(DA_ERR_ALIGN, "gradients must be aligned to their elements");
    size_t need = 0;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    bool had[2] = {false, false};
    for (int i = 0; i < a.sides; ++i) {
        da::QkrSide &s = a.side[i];
        had[s.keys] = true;
        s.g = s.keys ? grad_out_k : grad_out_q;
        s.grad_w = s.keys ? grad_k_weight : grad_q_weight;
        if (!s.y || !s.g) return da::fail(DA_ERR_NULL, "a gradient of q or k is NULL");
        if (s.w) {
            s.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + need);
            need += da::part_bytes(s);
        }
    }
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return da::fail(DA_ERR_WORKSPACE, "workspace of %zu bytes; %zu are needed", workspace ? workspace_bytes : size_t{0}, need);
        if (!da::aligned(workspace, 256)) return da::fail(DA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    }
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < 2 && e == cudaSuccess; ++i)  // no vectors: no gradient
        if (float *w = i ? grad_k_weight : grad_q_weight; w && !had[i]) e = cudaMemsetAsync(w, 0, sizeof(float) * p->width, cs);
    if (e == cudaSuccess && a.sides > 0) {
        const int V = da::plan_sides(a, elem, true);
        const unsigned grid = da::share_ctas(a, da::kBackwardCtas, 0);
        e = p->dtype == DA_F32    ? da::backward_pieces<float>(a, V, grid, cs)
            : p->dtype == DA_BF16 ? da::backward_pieces<__nv_bfloat16>(a, V, grid, cs)
                                  : da::backward_pieces<__half>(a, V, grid, cs);
        if (e == cudaSuccess && need > 0)
            e = da::launch_pdl(da::qkr_weight_kernel, dim3((p->width + 31) / 32, a.sides), dim3(1024), 0, cs, a);
    }
    return e == cudaSuccess ? DA_OK : da::cuda_fail(e, "rotary norm backward launch");
}

}  // extern "C"
