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
// floating point. Memory traffic bounds both passes.
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

template <typename T> __device__ __forceinline__ float qkr_float(T v);
template <> __device__ __forceinline__ float qkr_float(float v) { return v; }
template <> __device__ __forceinline__ float qkr_float(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float qkr_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T qkr_round(float v);
template <> __device__ __forceinline__ float qkr_round(float v) { return v; }
template <> __device__ __forceinline__ __half qkr_round(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 qkr_round(float v) { return __float2bfloat16_rn(v); }

// V channels as they lie in memory.
template <typename T, int V> union Piece {
    typename QkrRaw<static_cast<int>(sizeof(T)) * V>::type raw;
    T v[V];
    __device__ __forceinline__ Piece() {}
};

// A lane's two pieces of each of its slots: SPL slots, 2 V channels each.
template <typename T, int V> constexpr int kSlots = V >= 4 ? 1 : V == 2 ? 2 : 4;

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

// Cosine and sine of pos * turns / 2^64 of a turn: the product's quarter turn
// next to it exactly, the rest, at most an eighth of a turn, in fp32.
__device__ __forceinline__ float2 angle(int pos, int64_t turns)
{
    const uint64_t at = static_cast<uint64_t>(static_cast<int64_t>(pos)) * static_cast<uint64_t>(turns);
    const uint32_t quarter = static_cast<uint32_t>((at + (uint64_t{1} << 61)) >> 62);
    const int64_t rest = static_cast<int64_t>(at - (static_cast<uint64_t>(quarter) << 62));
    float s, c;
    sincospif(static_cast<float>(rest) * 0x1p-63f, &s, &c);
    if (quarter & 1) {
        const float t = c;
        c = -s;
        s = t;
    }
    return (quarter & 2) ? make_float2(-c, -s) : make_float2(c, s);
}

// Which token a warp's vectors are of, and where they lie.
struct Run {
    int64_t token0;
    int count;     // tokens
};

__device__ __forceinline__ void token_place(const QkrSide &s, int64_t token, int &b, int &l)
{
    b = static_cast<int>(s.div_L.div(static_cast<uint32_t>(token)));
    l = static_cast<int>(token - static_cast<int64_t>(b) * s.L);
}

__device__ __forceinline__ int position(const QkrArgs &a, const QkrSide &s, int64_t token)
{
    if (s.pos) return s.pos[token];
    int b, l;
    token_place(s, token, b, l);
    return static_cast<int>(static_cast<uint32_t>(a.lengths ? a.lengths[b] : s.first) + static_cast<uint32_t>(l));
}

// The angles of a run's tokens, [token][R / 2], times the magnitude.
__device__ __forceinline__ void fill_angles(const QkrArgs &a, const QkrSide &s, const Run &run, float2 *cs)
{
    const int hp = s.R / 2;
    for (int i = threadIdx.x & 31; i < run.count * hp; i += 32) {
        const int t = static_cast<int>(s.div_hp.div(i));
        const float2 v = angle(position(a, s, run.token0 + t), a.turns[i - t * hp]);
        cs[i] = make_float2(v.x * a.magnitude, v.y * a.magnitude);
    }
}

// z_a, z_b of the pairs of a slot; back: the turn in the other direction.
template <int V, bool BACK>
__device__ __forceinline__ void turn(const float2 *cs, int interleaved, float (&a)[V], float (&b)[V])
{
    if (V > 1 && interleaved) {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            if constexpr (V > 1) {
                const float2 u = cs[j / 2], v = cs[V / 2 + j / 2];
                const float us = BACK ? -u.y : u.y, vs = BACK ? -v.y : v.y;
                const float a0 = a[j], a1 = a[j + 1], b0 = b[j], b1 = b[j + 1];
                a[j] = a0 * u.x - a1 * us;
                a[j + 1] = a0 * us + a1 * u.x;
                b[j] = b0 * v.x - b1 * vs;
                b[j + 1] = b0 * vs + b1 * v.x;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float2 u = cs[j];
            const float us = BACK ? -u.y : u.y, x = a[j], y = b[j];
            a[j] = x * u.x - y * us;
            b[j] = x * us + y * u.x;
        }
    }
}

__device__ __forceinline__ float lanes_sum(float v, int sg_log2)
{
    for (int o = 1 << sg_log2 >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename T, int V> __device__ __forceinline__ Piece<T, V> load_piece(const T *base, int at)
{
    Piece<T, V> p;
    p.raw = __ldcs(reinterpret_cast<const decltype(p.raw) *>(base + at));
    return p;
}

// ---- forward, and append ---------------------------------------------------

// Vectors that a group of lanes has under way at once.
constexpr int kAhead = 2;

template <typename T, int V, bool PAGED>
__global__ void __launch_bounds__(kQkrThreads) qkr_forward_kernel(const __grid_constant__ QkrArgs a)
{
    constexpr int SPL = kSlots<T, V>;
    __shared__ __align__(16) float2 all_cs[kQkrWarps][kPairs];
    __shared__ int2 all_where[PAGED ? kQkrWarps : 1][kTokens];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kQkrWarps + warp;
    int which = 0;
    while (which + 1 < a.sides && unit >= a.side[which + 1].unit0) ++which;
    const QkrSide &s = a.side[which];
    Run run;
    run.token0 = (unit - s.unit0) * s.tpw;
    if (run.token0 >= s.tokens) return;
    run.count = static_cast<int>(min(static_cast<int64_t>(s.tpw), s.tokens - run.token0));
    float2 *cs = all_cs[warp];

    const int lanes = 1 << s.sg_log2, sub = lane >> s.sg_log2, step = 32 >> s.sg_log2;
    const int HM = s.H * s.M, vectors = run.count * HM;
    Slot slot[SPL];
    float wa[SPL][V], wb[SPL][V];
#pragma unroll
    for (int p = 0; p < SPL; ++p) {
        slot[p] = slot_of<V>(s, (lane & (lanes - 1)) + p * 32, a.interleaved);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            wa[p][j] = s.w && slot[p].a >= 0 ? s.w[slot[p].a + j] : 1.f;
            wb[p][j] = s.w && slot[p].b >= 0 ? s.w[slot[p].b + j] : 1.f;
        }
    }
    Piece<T, V> xa[kAhead][SPL], xb[kAhead][SPL];
    int64_t to[kAhead];  // where the vector goes, or -1
    const auto fetch = [&](int i0) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u * step;
            to[u] = -1;
            if (i >= vectors) continue;
            const int t = static_cast<int>(s.div_vec.div(i)), hm = i - t * HM, h = s.M == 2 ? hm >> 1 : hm, m = s.M == 2 ? hm & 1 : 0;
            int b, l;
            token_place(s, run.token0 + t, b, l);
            const T *x = static_cast<const T *>(s.x) + b * s.xs[0] + l * s.xs[1] + h * s.xs[2] + m * s.xs[3];
#pragma unroll
            for (int p = 0; p < SPL; ++p) {
                if (slot[p].a >= 0) xa[u][p] = load_piece<T, V>(x, slot[p].a);
                if (slot[p].b >= 0) xb[u][p] = load_piece<T, V>(x, slot[p].b);
            }
            to[u] = b * s.ys[0] + l * s.ys[1] + h * s.ys[2] + m * s.ys[3];
        }
    };
    fetch(sub);

    fill_angles(a, s, run, cs);
    if (PAGED && s.paged && lane < run.count) {
        int b, l;
        token_place(s, run.token0 + lane, b, l);
        int2 at = make_int2(-1, 0);
        const int64_t place = static_cast<int64_t>(a.lengths[b]) + l;
        const int count = a.counts ? a.counts[b] : s.L;
        if (l < count && place >= 0 && place < static_cast<int64_t>(a.table_pages) * a.page_size) {
            const int n = static_cast<int>(a.div_page.div(static_cast<uint32_t>(place)));
            const int page = a.table[static_cast<int64_t>(b) * a.table_pages + n];
            if (page >= 0 && page < a.num_pages) at = make_int2(page, static_cast<int>(place) - n * a.page_size);
        }
        all_where[warp][lane] = at;
    }
    __syncwarp();

    for (int i0 = sub; i0 - sub < vectors; i0 += kAhead * step) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u * step;
            const bool live = to[u] >= 0;
            const int t = live ? static_cast<int>(s.div_vec.div(i)) : 0;
            float fa[SPL][V], fb[SPL][V];
            float sq = 0.f;
#pragma unroll
            for (int p = 0; p < SPL; ++p)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    fa[p][j] = live && slot[p].a >= 0 ? qkr_float(xa[u][p].v[j]) : 0.f;
                    fb[p][j] = live && slot[p].b >= 0 ? qkr_float(xb[u][p].v[j]) : 0.f;
                    sq = fmaf(fa[p][j], fa[p][j], sq);
                    sq = fmaf(fb[p][j], fb[p][j], sq);
                }
            if (s.normed) {
                const float r = rsqrtf(fmaf(lanes_sum(sq, s.sg_log2), s.inv_D, a.eps));
#pragma unroll
                for (int p = 0; p < SPL; ++p)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        fa[p][j] = fa[p][j] * r * wa[p][j];
                        fb[p][j] = fb[p][j] * r * wb[p][j];
                    }
            }
            if (!live) continue;
            int64_t at = to[u];
            if (PAGED && s.paged) {
                const int2 w = all_where[warp][t];
                if (w.x < 0) continue;
                const int hm = i - t * HM, h = s.M == 2 ? hm >> 1 : hm, m = s.M == 2 ? hm & 1 : 0;
                at = w.x * s.ys[0] + w.y * s.ys[1] + h * s.ys[2] + m * s.ys[3];
            }
            T *y = static_cast<T *>(s.y) + at;
#pragma unroll
            for (int p = 0; p < SPL; ++p) {
                if (slot[p].pair >= 0) turn<V, false>(cs + t * (s.R / 2) + slot[p].pair, a.interleaved, fa[p], fb[p]);
                Piece<T, V> oa, ob;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    oa.v[j] = qkr_round<T>(fa[p][j]);
                    ob.v[j] = qkr_round<T>(fb[p][j]);
                }
                if (slot[p].a >= 0) *reinterpret_cast<decltype(oa.raw) *>(y + slot[p].a) = oa.raw;
                if (slot[p].b >= 0) *reinterpret_cast<decltype(ob.raw) *>(y + slot[p].b) = ob.raw;
            }
        }
        fetch(i0 + kAhead * step);
    }
}

// ---- backward --------------------------------------------------------------

// CTAs of a side walk over its runs; every lane sums its channels' part of the
// weight's gradient over all of its vectors in registers, and a CTA leaves one
// row of sums.
template <typename T, int V>
__global__ void __launch_bounds__(kQkrThreads) qkr_backward_kernel(const __grid_constant__ QkrArgs a)
{
    constexpr int SPL = kSlots<T, V>;
    __shared__ __align__(16) float2 all_cs[kQkrWarps][kPairs];
    __shared__ float sums[kQkrWarps][QKR_MAX_WIDTH];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int which = 0;
    while (which + 1 < a.sides && static_cast<int64_t>(blockIdx.x) >= a.side[which + 1].unit0) ++which;
    const QkrSide &s = a.side[which];
    const int cta = static_cast<int>(blockIdx.x - s.unit0);
    float2 *cs = all_cs[warp];
    const int lanes = 1 << s.sg_log2, sub = lane >> s.sg_log2, step = 32 >> s.sg_log2, HM = s.H * s.M;
    Slot slot[SPL];
    float wa[SPL][V], wb[SPL][V], ga[SPL][V], gb[SPL][V];
#pragma unroll
    for (int p = 0; p < SPL; ++p) {
        slot[p] = slot_of<V>(s, (lane & (lanes - 1)) + p * 32, a.interleaved);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            wa[p][j] = s.w && slot[p].a >= 0 ? s.w[slot[p].a + j] : 1.f;
            wb[p][j] = s.w && slot[p].b >= 0 ? s.w[slot[p].b + j] : 1.f;
            ga[p][j] = gb[p][j] = 0.f;
        }
    }
    for (int64_t r = static_cast<int64_t>(cta) * kQkrWarps + warp; r * s.tpw < s.tokens; r += static_cast<int64_t>(s.units) * kQkrWarps) {
        Run run;
        run.token0 = r * s.tpw;
        run.count = static_cast<int>(min(static_cast<int64_t>(s.tpw), s.tokens - run.token0));
        const int vectors = run.count * HM;
        Piece<T, V> xa[kAhead][SPL], xb[kAhead][SPL], za[kAhead][SPL], zb[kAhead][SPL];
        int64_t to[kAhead];
        const auto fetch = [&](int i0) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = i0 + u * step;
                to[u] = -1;
                if (i >= vectors) continue;
                const int t = static_cast<int>(s.div_vec.div(i)), hm = i - t * HM;
                int b, l;
                token_place(s, run.token0 + t, b, l);
                const T *x = static_cast<const T *>(s.x) + b * s.xs[0] + l * s.xs[1] + (hm >> 1) * s.xs[2] + (hm & 1) * s.xs[3];
                to[u] = (run.token0 * HM + i) * s.D;
                const T *g = static_cast<const T *>(s.g) + to[u];
#pragma unroll
                for (int p = 0; p < SPL; ++p) {
                    if (slot[p].a >= 0) {
                        za[u][p] = load_piece<T, V>(g, slot[p].a);
                        if (s.normed) xa[u][p] = load_piece<T, V>(x, slot[p].a);
                    }
                    if (slot[p].b >= 0) {
                        zb[u][p] = load_piece<T, V>(g, slot[p].b);
                        if (s.normed) xb[u][p] = load_piece<T, V>(x, slot[p].b);
                    }
                }
            }
        };
        fetch(sub);
        __syncwarp();  // the run before has been read
        fill_angles(a, s, run, cs);
        __syncwarp();
        for (int i0 = sub; i0 - sub < vectors; i0 += kAhead * step) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = i0 + u * step;
                const bool live = to[u] >= 0;
                const int t = live ? static_cast<int>(s.div_vec.div(i)) : 0;
                float ha[SPL][V], hb[SPL][V];
#pragma unroll
                for (int p = 0; p < SPL; ++p) {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        ha[p][j] = live && slot[p].a >= 0 ? qkr_float(za[u][p].v[j]) : 0.f;
                        hb[p][j] = live && slot[p].b >= 0 ? qkr_float(zb[u][p].v[j]) : 0.f;
                    }
                    if (slot[p].pair >= 0 && live) turn<V, true>(cs + t * (s.R / 2) + slot[p].pair, a.interleaved, ha[p], hb[p]);
                }
                if (s.normed) {
                    float na[SPL][V], nb[SPL][V], sq = 0.f;
#pragma unroll
                    for (int p = 0; p < SPL; ++p)
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            na[p][j] = live && slot[p].a >= 0 ? qkr_float(xa[u][p].v[j]) : 0.f;
                            nb[p][j] = live && slot[p].b >= 0 ? qkr_float(xb[u][p].v[j]) : 0.f;
                            sq = fmaf(na[p][j], na[p][j], sq);
                            sq = fmaf(nb[p][j], nb[p][j], sq);
                        }
                    const float rn = rsqrtf(fmaf(lanes_sum(sq, s.sg_log2), s.inv_D, a.eps));
                    float dot = 0.f;
#pragma unroll
                    for (int p = 0; p < SPL; ++p)
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            na[p][j] *= rn;
                            nb[p][j] *= rn;
                            ga[p][j] = fmaf(ha[p][j], na[p][j], ga[p][j]);
                            gb[p][j] = fmaf(hb[p][j], nb[p][j], gb[p][j]);
                            ha[p][j] *= wa[p][j];
                            hb[p][j] *= wb[p][j];
                            dot = fmaf(ha[p][j], na[p][j], dot);
                            dot = fmaf(hb[p][j], nb[p][j], dot);
                        }
                    const float mean = lanes_sum(dot, s.sg_log2) * s.inv_D;
#pragma unroll
                    for (int p = 0; p < SPL; ++p)
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            ha[p][j] = rn * fmaf(-na[p][j], mean, ha[p][j]);
                            hb[p][j] = rn * fmaf(-nb[p][j], mean, hb[p][j]);
                        }
                }
                if (!live) continue;
                T *y = static_cast<T *>(s.y) + to[u];
#pragma unroll
                for (int p = 0; p < SPL; ++p) {
                    Piece<T, V> oa, ob;
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        oa.v[j] = qkr_round<T>(ha[p][j]);
                        ob.v[j] = qkr_round<T>(hb[p][j]);
                    }
                    if (slot[p].a >= 0) *reinterpret_cast<decltype(oa.raw) *>(y + slot[p].a) = oa.raw;
                    if (slot[p].b >= 0) *reinterpret_cast<decltype(ob.raw) *>(y + slot[p].b) = ob.raw;
                }
            }
            fetch(i0 + kAhead * step);
        }
    }
    if (!s.part) return;
#pragma unroll
    for (int p = 0; p < SPL; ++p)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            for (int o = lanes; o < 32; o <<= 1) {
                ga[p][j] += __shfl_xor_sync(0xffffffffu, ga[p][j], o);
                gb[p][j] += __shfl_xor_sync(0xffffffffu, gb[p][j], o);
            }
            if (sub == 0) {
                if (slot[p].a >= 0) sums[warp][slot[p].a + j] = ga[p][j];
                if (slot[p].b >= 0) sums[warp][slot[p].b + j] = gb[p][j];
            }
        }
    __syncthreads();
    for (int d = threadIdx.x; d < s.D; d += kQkrThreads) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < kQkrWarps; ++w) t += sums[w][d];
        s.part[static_cast<int64_t>(cta) * s.D + d] = t;
    }
}

// grad_weight of a side: the CTAs' rows in a fixed order, one warp per channel.
__global__ void __launch_bounds__(kQkrThreads) qkr_weight_kernel(const __grid_constant__ QkrArgs a)
{
    pdl_wait();
    const QkrSide &s = a.side[blockIdx.y];
    const int d = blockIdx.x * kQkrWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (!s.part || d >= s.D) return;
    float t = 0.f;
    for (int c = lane; c < s.units; c += 32) t += s.part[static_cast<int64_t>(c) * s.D + d];
    t = lanes_sum(t, 5);
    if (lane == 0) s.grad_w[d] = t;
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

constexpr int kBackwardCtas = 152 * 4;  // of both sides together

// Units of each side, in proportion to its vectors.
void backward_units(QkrArgs &a)
{
    int64_t all = 0, unit = 0;
    for (int i = 0; i < a.sides; ++i) all += a.side[i].tokens * a.side[i].H;
    for (int i = 0; i < a.sides; ++i) {
        QkrSide &s = a.side[i];
        const int64_t runs = (s.tokens + static_cast<int64_t>(s.tpw) * kQkrWarps - 1) / (static_cast<int64_t>(s.tpw) * kQkrWarps);
        int64_t n = static_cast<int64_t>(static_cast<double>(kBackwardCtas) * s.tokens * s.H / all);
        n = n < 1 ? 1 : n;
        s.units = static_cast<int32_t>(n < runs ? n : runs);
        s.unit0 = unit;
        unit += s.units;
    }
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
    int64_t units = 0;
    for (int i = 0; i < a.sides; ++i) {
        a.side[i].unit0 = units;
        units += (a.side[i].tokens + a.side[i].tpw - 1) / a.side[i].tpw;
    }
    const unsigned grid = static_cast<unsigned>((units + kQkrWarps - 1) / kQkrWarps);
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
        da::backward_units(a);
        const da::QkrSide &last = a.side[a.sides - 1];
        const unsigned grid = static_cast<unsigned>(last.unit0 + last.units);
        e = p->dtype == DA_F32    ? da::backward_pieces<float>(a, V, grid, cs)
            : p->dtype == DA_BF16 ? da::backward_pieces<__nv_bfloat16>(a, V, grid, cs)
                                  : da::backward_pieces<__half>(a, V, grid, cs);
        if (e == cudaSuccess && need > 0)
            e = da::launch_pdl(da::qkr_weight_kernel, dim3((p->width + da::kQkrWarps - 1) / da::kQkrWarps, a.sides),
                               dim3(da::kQkrThreads), 0, cs, a);
    }
    return e == cudaSuccess ? DA_OK : da::cuda_fail(e, "rotary norm backward launch");
}

}  // extern "C"
