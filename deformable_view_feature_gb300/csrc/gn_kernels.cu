// Group norm with an activation over packed channels-last maps (include/gn.h).
//
// A map is cut into tiles of `tr` rows, and each pass is one kernel of two
// CTAs per tile, ordered by a ticket that a CTA draws when it starts: first a
// tile's sums, and some hundred tiles later, when its map's sums are complete,
// the same tile's outputs. That distance keeps what lies between in the 129 MB
// L2, so the second reading of a tile comes from there and device memory is
// read once. In between, CTAs of their own join the map's sums, in a fixed
// order. A CTA's threads form a grid of 4-channel columns
// x rows of its tile, so every access is a full row segment and a thread keeps
// its channels' parameters in registers; it sends its first loads before it
// waits for anything. 6 x 89,760 rows of 256 fp32 channels: 235 us forward and
// 439 backward, 4.7 and 3.8 TB/s of what has to be moved (three launches, each
// reading everything: 289 and 577).
//
// The wait for a map's sums cannot stall: a CTA that waits has a later ticket
// than every tile it waits for, and those, already running, are summed without
// waiting. It is bounded all the same; a wait that ran out turns what depended
// on it into NaN and sets a word that gn_device_status reads.
//
// Forward statistics: a thread takes the rows of a batch about their own mean,
// while they are in registers, and batches, the tile's threads, its channels
// and at last the tiles are joined by
//   M2 = sum M2_t + sum n_t (mean_t - mean)^2.
// No sum of squares about another value occurs, so neither a mean far larger
// than the spread nor a row unlike the rest costs digits.
#include <atomic>
#include <cmath>
#include <cuda_bf16.h>

#include "da_internal.cuh"
#include "gn.h"

namespace da {
namespace {

constexpr int kGnThreads = 256;
constexpr int kGnCtas = 3;         // resident per SM: up to 85 registers a thread
constexpr int kGnSmall = 65536;    // bytes of a map that one CTA takes alone
constexpr int kGnTries = 1 << 22;  // of a wait, about a microsecond each at most (da_gn_wait_tries)

std::atomic<int32_t> g_gn_tries{kGnTries};

struct GnMap {
    int32_t rows, start;  // pixels, first feature row
    int32_t tile0;        // its first tile among the batch item's tiles
    int32_t scale;        // s of (k, s)
};

struct GnArgs {
    const void *x, *g;   // feat, grad_out
    void *y;             // out, or grad_feat
    const float *gamma, *beta;
    float *stats;        // [B, maps, G, 2]
    float *part;         // per tile: forward [G, 2] mean, M2; backward [2, C] sums of h and h*n
    float *sums;         // backward: [B, maps, 2, C]
    float *group;        // backward: [B, maps, G, 2] mean(gamma*h), mean(gamma*h*n)
    float *grad_gamma, *grad_beta;
    // Counters, zero at launch: tickets drawn, joins done or left out, whether
    // one was left out, then per (batch item, map) tiles summed and joins done.
    uint32_t *tickets, *all_done, *left_out, *tiles_done, *ready;
    int32_t tries;       // of a wait
    int32_t ntiles, lag; // tiles in all, tiles between a tile's sums and its outputs
    int32_t joins;       // CTAs that share a map's join
    int64_t rows;        // per batch item
    int32_t B, C, G, Cg, nmaps, S, tiles, tr, affine_scales;
    FastDiv div_Cg;
    float eps;
    GnMap maps[DA_MAX_MAPS];
};

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f(float v) { return v; }
template <> __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f(float v) { return v; }
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

// V consecutive channels as they are loaded: four (16 or 8 bytes), or one
// where rows are not multiples of 16 bytes.
template <int BYTES> struct Raw;
template <> struct Raw<16> { using type = uint4; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<2> { using type = unsigned short; };
template <typename T, int V> using Pack = typename Raw<static_cast<int>(sizeof(T)) * V>::type;

__device__ __forceinline__ void two(uint32_t w, float &a, float &b, const __nv_bfloat16 *)
{
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void two(uint32_t w, float &a, float &b, const __half *)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    a = f.x;
    b = f.y;
}
__device__ __forceinline__ uint32_t two(float a, float b, const __nv_bfloat16 *)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t two(float a, float b, const __half *)
{
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <typename T, int V> __device__ __forceinline__ void unpack(const Pack<T, V> &p, float (&f)[V])
{
    if constexpr (V == 1) {
        f[0] = to_f(*reinterpret_cast<const T *>(&p));
    } else if constexpr (sizeof(T) == 4) {
        f[0] = __uint_as_float(p.x);
        f[1] = __uint_as_float(p.y);
        f[2] = __uint_as_float(p.z);
        f[3] = __uint_as_float(p.w);
    } else {
        two(p.x, f[0], f[1], static_cast<const T *>(nullptr));
        two(p.y, f[2], f[3], static_cast<const T *>(nullptr));
    }
}

// LAST: the data's last use, so that it leaves the caches first, like what is
// stored.
template <typename T, int V, bool LAST> __device__ __forceinline__ Pack<T, V> load_pack(const T *base, int at)
{
    const auto *p = reinterpret_cast<const Pack<T, V> *>(base + at);
    return LAST ? __ldcs(p) : __ldcg(p);
}

template <typename T, int V> __device__ __forceinline__ void store_row(void *base, int64_t at, const float (&f)[V])
{
    Pack<T, V> p;
    if constexpr (V == 1) {
        const T v = from_f<T>(f[0]);
        p = *reinterpret_cast<const Pack<T, V> *>(&v);
    } else if constexpr (sizeof(T) == 4) {
        p = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    } else {
        p = make_uint2(two(f[0], f[1], static_cast<const T *>(nullptr)), two(f[2], f[3], static_cast<const T *>(nullptr)));
    }
    __stcs(reinterpret_cast<Pack<T, V> *>(static_cast<T *>(base) + at), p);
}

// 1 / (1 + exp(-z)) by the hardware's 2^x and reciprocal (each within a few
// units in the last place); exp(-z) past the largest number gives 0.
__device__ __forceinline__ float logistic(float z)
{
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}

// act(z), and act'(z) for the backward pass.
template <int ACT> __device__ __forceinline__ float act_of(float z)
{
    if (ACT == GN_ACT_RELU) return z < 0.f ? 0.f : z;  // NaN stays NaN
    if (ACT == GN_ACT_SILU) return z * logistic(z);
    return z;
}
template <int ACT> __device__ __forceinline__ float act_slope(float z)
{
    if (ACT == GN_ACT_RELU) return z > 0.f ? 1.f : 0.f;
    if (ACT == GN_ACT_SILU) {
        const float s = logistic(z);
        return fmaf(z * s, 1.f - s, s);
    }
    return 1.f;
}

struct Tile {
    int b, map;
    int64_t row;  // first row, over all batch items
    int rows;
};

__device__ __forceinline__ Tile find_tile(const GnArgs &a, int id)
{
    Tile t;
    t.b = id / a.tiles;
    const int in = id - t.b * a.tiles;
    int lo = 0, hi = a.nmaps - 1;
    while (lo < hi) {  // the last map whose first tile is at or before `in`
        const int mid = (lo + hi + 1) >> 1;
        if (a.maps[mid].tile0 <= in) lo = mid; else hi = mid - 1;
    }
    t.map = lo;
    const int off = (in - a.maps[lo].tile0) * a.tr;
    t.rows = min(a.tr, a.maps[lo].rows - off);
    t.row = static_cast<int64_t>(t.b) * a.rows + a.maps[lo].start + off;
    return t;
}

// How the CTA's threads cover a tile: column `col` of each block of `cols`
// columns, rows lane, lane + lanes, ...; a thread past cols * lanes is idle.
struct Cover {
    int ncols, cols, lanes, col, lane;
    bool on;
};

template <int V> __device__ __forceinline__ Cover cover(int C)
{
    Cover c;
    c.ncols = C / V;
    c.cols = min(c.ncols, kGnThreads);
    c.lanes = kGnThreads / c.cols;
    c.lane = threadIdx.x / c.cols;
    c.col = threadIdx.x - c.lane * c.cols;
    c.on = c.lane < c.lanes;
    return c;
}

// The lane's rows of a tile, U at a time; of one tensor, or of two at the same
// places (if TWO). begin() sends the first loads, which need nothing but the
// tile, ahead of whatever else the CTA has to wait for; batches() then calls
// use() for every U rows, there(u) of which are in p and q, and each()
// use(offset from the column's place in the tile's first row, x, g) per row.
template <typename T, int V, bool TWO, bool LAST, int U> struct Rows {
    Pack<T, V> p[U], q[TWO ? U : 1];
    const T *px, *pg;
    int o, step, end;

    __device__ __forceinline__ void load()
    {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (there(u)) {
                p[u] = load_pack<T, V, LAST>(px, o + u * step);
                if (TWO) q[u] = load_pack<T, V, LAST>(pg, o + u * step);
            }
    }
    __device__ __forceinline__ void begin(const Cover &c, bool on, int rows, int C, const void *x, const void *g, int64_t at)
    {
        px = static_cast<const T *>(x) + at;
        pg = static_cast<const T *>(g) + at;
        step = c.lanes * C;
        o = c.lane * C;
        end = on ? rows * C : 0;
        load();
    }
    __device__ __forceinline__ bool there(int u) const { return o + u * step < end; }
    template <typename Use> __device__ __forceinline__ void batches(Use use)
    {
        while (o < end) {
            use();
            o += U * step;
            load();
        }
    }
    template <typename Use> __device__ __forceinline__ void each(Use use)
    {
        batches([&] {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (there(u)) {
                    float v[V], h[V];
                    unpack<T, V>(p[u], v);
                    if (TWO) unpack<T, V>(q[u], h);
                    use(o + u * step, v, h);
                }
        });
    }
};

// Rows to a batch: 128 bytes of x, or 64 of x and grad_out each, to a thread.
template <typename T, int V> constexpr int kFwdRows = V == 1 ? 8 : 128 / (V * static_cast<int>(sizeof(T)));
template <typename T, int V> constexpr int kBwdRows = V == 1 ? 4 : 64 / (V * static_cast<int>(sizeof(T)));

// Sums over the row lanes of two values per channel, in the order of the
// lanes. The sums of channel i of column c are left in scratch[c*V + i] and
// scratch[second + c*V + i], second = lanes * cols * V.
template <int V>
__device__ __forceinline__ void lane_sums(const Cover &c, const float (&p)[V], const float (&q)[V], float *scratch)
{
    const int w = c.cols * V;
    if (c.on) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            scratch[c.lane * w + c.col * V + i] = p[i];
            scratch[(c.lanes + c.lane) * w + c.col * V + i] = q[i];
        }
    }
    __syncthreads();
    for (int ch = threadIdx.x; ch < 2 * w; ch += kGnThreads) {
        const int which = ch >= w;
        float *at = scratch + which * c.lanes * w + (ch - which * w);
        float s = at[0];
        for (int l = 1; l < c.lanes; ++l) s += at[l * w];
        at[0] = s;  // no other thread reads this channel's column
    }
    __syncthreads();
}

// ---- forward ---------------------------------------------------------------

template <typename T, int V> __device__ void tile_stats(const GnArgs &a, const Tile &t, int id, float *smem)
{
    float *scratch = smem;                               // [2][lanes][cols*V] <= 2 * kGnThreads * V
    float *mean_c = smem + 2 * kGnThreads * V, *m2_c = mean_c + a.C;
    const Cover c = cover<V>(a.C);
    constexpr int U = kFwdRows<T, V>;
    // A batch's mean comes from sums about its first row, except in 16 bits:
    // 16 such values of one magnitude sum exactly in fp32 as they are.
    constexpr bool pivot = sizeof(T) == 4;
    for (int c0 = 0; c0 < c.ncols; c0 += c.cols) {
        const int col = c0 + c.col;
        const bool on = c.on && col < c.ncols;
        const int64_t at = t.row * a.C + static_cast<int64_t>(on ? col : 0) * V;
        Rows<T, V, false, false, U> rows;
        rows.begin(c, on, t.rows, a.C, a.x, a.x, at);
        // Lane l of the rows has `each` of them, or one more.
        const int each = t.rows / c.lanes, more = t.rows - each * c.lanes;
        float mean[V], m2[V], count = 0.f;
        int left = each + (c.lane < more);
#pragma unroll
        for (int i = 0; i < V; ++i) mean[i] = m2[i] = 0.f;
        rows.batches([&] {
            float v[V], first[V], s[V], q[V];
            const auto add = [&](int u) {
                unpack<T, V>(rows.p[u], v);
#pragma unroll
                for (int i = 0; i < V; ++i) s[i] += pivot ? v[i] - first[i] : v[i];
            };
            const auto square = [&](int u) {
                unpack<T, V>(rows.p[u], v);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float d = v[i] - s[i];
                    q[i] = fmaf(d, d, q[i]);
                }
            };
            if (pivot) unpack<T, V>(rows.p[0], first);
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] = q[i] = 0.f;
            const float n = static_cast<float>(min(left, U)), inv = __fdividef(1.f, n), share = __fdividef(n, count + n);
            const auto means = [&] {
#pragma unroll
                for (int i = 0; i < V; ++i) s[i] = pivot ? fmaf(s[i], inv, first[i]) : s[i] * inv;
            };
            if (left >= U) {
#pragma unroll
                for (int u = 0; u < U; ++u) add(u);
                means();
#pragma unroll
                for (int u = 0; u < U; ++u) square(u);
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (u < left) add(u);
                means();
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (u < left) square(u);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = s[i] - mean[i];
                mean[i] = fmaf(d, share, mean[i]);
                m2[i] += q[i] + d * d * (count * share);
            }
            count += n;
            left -= U;
        });
        const int w = c.cols * V, second = c.lanes * w;
        if (c.on) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                scratch[c.lane * w + c.col * V + i] = mean[i];
                scratch[second + c.lane * w + c.col * V + i] = m2[i];
            }
        }
        __syncthreads();
        const int lanes = min(c.lanes, t.rows);
        for (int ch = threadIdx.x; ch < min(c.cols, c.ncols - c0) * V; ch += kGnThreads) {
            const float m0 = scratch[ch];
            float s = 0.f, q = 0.f;
            for (int l = 1; l < lanes; ++l) s = fmaf(static_cast<float>(each + (l < more)), scratch[l * w + ch] - m0, s);
            const float m = m0 + s / static_cast<float>(t.rows);
            for (int l = 0; l < lanes; ++l) {
                const float d = scratch[l * w + ch] - m;
                q += fmaf(static_cast<float>(each + (l < more)) * d, d, scratch[second + l * w + ch]);
            }
            mean_c[c0 * V + ch] = m;
            m2_c[c0 * V + ch] = q;
        }
        __syncthreads();
    }
    for (int g = threadIdx.x; g < a.G; g += kGnThreads) {
        float m = 0.f;
        for (int i = 0; i < a.Cg; ++i) m += mean_c[g * a.Cg + i];
        m /= static_cast<float>(a.Cg);
        float s = 0.f, d2 = 0.f;
        for (int i = 0; i < a.Cg; ++i) {
            const float d = mean_c[g * a.Cg + i] - m;
            s += m2_c[g * a.Cg + i];
            d2 = fmaf(d, d, d2);
        }
        float *o = a.part + (static_cast<int64_t>(id) * a.G + g) * 2;
        o[0] = m;
        o[1] = s + static_cast<float>(t.rows) * d2;
    }
}

// The groups' statistics of a map from its tiles' means and squared
// deviations: `lanes` threads per group take every lanes-th tile each, then
// the lanes in order.
__device__ void join_stats(const GnArgs &a, int b, int map, float *smem)
{
    const GnMap m = a.maps[map];
    const int n = (m.rows + a.tr - 1) / a.tr, tid = threadIdx.x;
    const float2 *part = reinterpret_cast<const float2 *>(a.part) + (static_cast<int64_t>(b) * a.tiles + m.tile0) * a.G;
    float2 *out = reinterpret_cast<float2 *>(a.stats) + (static_cast<int64_t>(b) * a.nmaps + map) * a.G;
    for (int g0 = 0; g0 < a.G; g0 += kGnThreads) {
        const int w = min(a.G - g0, kGnThreads), lanes = kGnThreads / w, lane = tid / w, g = g0 + tid - lane * w;
        float mean = 0.f, m2 = 0.f, count = 0.f;
        if (lane < lanes)
            for (int t = lane; t < n; t += 8 * lanes) {
                float2 p[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (t + u * lanes < n) p[u] = __ldcg(part + static_cast<int64_t>(t + u * lanes) * a.G + g);
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (t + u * lanes < n) {
                        const float k = static_cast<float>(min(a.tr, m.rows - (t + u * lanes) * a.tr)), d = p[u].x - mean;
                        const float share = k / (count + k);
                        mean = fmaf(d, share, mean);
                        m2 += p[u].y + d * d * (count * share) * static_cast<float>(a.Cg);
                        count += k;
                    }
            }
        smem[tid] = mean;
        smem[kGnThreads + tid] = m2;
        smem[2 * kGnThreads + tid] = count;
        __syncthreads();
        if (tid < w) {
            for (int l = 1; l < lanes; ++l) {
                const float k = smem[2 * kGnThreads + l * w + tid];
                if (k == 0.f) break;
                const float d = smem[l * w + tid] - mean, share = k / (count + k);
                mean = fmaf(d, share, mean);
                m2 += smem[kGnThreads + l * w + tid] + d * d * (count * share) * static_cast<float>(a.Cg);
                count += k;
            }
            out[g] = make_float2(mean, 1.f / sqrtf(m2 / (count * static_cast<float>(a.Cg)) + a.eps));
        }
        __syncthreads();
    }
}

// In the place of a join that its tiles' sums did not reach in time.
__device__ void nan_stats(const GnArgs &a, int b, int map)
{
    float *out = a.stats + (static_cast<int64_t>(b) * a.nmaps + map) * a.G * 2;
    for (int i = threadIdx.x; i < 2 * a.G; i += kGnThreads) out[i] = NAN;
}

template <typename T, int V> __device__ void tile_nan(const GnArgs &a, const Tile &t)
{
    float nan[V];
#pragma unroll
    for (int i = 0; i < V; ++i) nan[i] = NAN;
    for (int i = threadIdx.x; i < t.rows * (a.C / V); i += kGnThreads) store_row<T, V>(a.y, t.row * a.C + static_cast<int64_t>(i) * V, nan);
}

template <typename T, int V, int ACT, typename Ready> __device__ void tile_apply(const GnArgs &a, const Tile &t, Ready ready)
{
    const Cover c = cover<V>(a.C);
    const float *st = a.stats + (static_cast<int64_t>(t.b) * a.nmaps + t.map) * a.G * 2;
    const int aff = a.affine_scales ? a.maps[t.map].scale * a.C : 0;
    for (int c0 = 0; c0 < c.ncols; c0 += c.cols) {
        const int col = c0 + c.col;
        const bool on = c.on && col < c.ncols;
        const int64_t at = t.row * a.C + static_cast<int64_t>(on ? col : 0) * V;
        Rows<T, V, false, true, kFwdRows<T, V>> rows;
        rows.begin(c, on, t.rows, a.C, a.x, a.x, at);
        float mean[V], mul[V], add[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int ch = (on ? col : 0) * V + i;
            mul[i] = a.gamma[aff + ch];
            add[i] = a.beta[aff + ch];
        }
        if (c0 == 0 && !ready()) return tile_nan<T, V>(a, t);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int g = static_cast<int>(a.div_Cg.div((on ? col : 0) * V + i));
            const float2 ms = __ldcg(reinterpret_cast<const float2 *>(st) + g);
            mean[i] = ms.x;
            mul[i] *= ms.y;
        }
        rows.each([&](int o, float (&v)[V], const float (&)[V]) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = act_of<ACT>(fmaf(v[i] - mean[i], mul[i], add[i]));
            store_row<T, V>(a.y, at + o, v);
        });
    }
}

// ---- backward --------------------------------------------------------------

// Sums of h and h*n per channel of the tile.
template <typename T, int V, int ACT> __device__ void tile_sums(const GnArgs &a, const Tile &t, int id, float *smem)
{
    const Cover c = cover<V>(a.C);
    const float *st = a.stats + (static_cast<int64_t>(t.b) * a.nmaps + t.map) * a.G * 2;
    const int aff = a.affine_scales ? a.maps[t.map].scale * a.C : 0;
    float *part = a.part + static_cast<int64_t>(id) * 2 * a.C;
    for (int c0 = 0; c0 < c.ncols; c0 += c.cols) {
        const int col = c0 + c.col;
        const bool on = c.on && col < c.ncols;
        const int64_t at = t.row * a.C + static_cast<int64_t>(on ? col : 0) * V;
        Rows<T, V, true, false, kBwdRows<T, V>> rows;
        rows.begin(c, on, t.rows, a.C, a.x, a.g, at);
        float p[V], q[V], mean[V], rstd[V], gam[V], bet[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int ch = (on ? col : 0) * V + i, g = static_cast<int>(a.div_Cg.div(ch));
            const float2 ms = __ldg(reinterpret_cast<const float2 *>(st) + g);
            mean[i] = ms.x;
            rstd[i] = ms.y;
            gam[i] = a.gamma[aff + ch];
            bet[i] = a.beta[aff + ch];
            p[i] = q[i] = 0.f;
        }
        rows.each([&](int, const float (&v)[V], const float (&h)[V]) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float n = (v[i] - mean[i]) * rstd[i];
                const float d = h[i] * act_slope<ACT>(fmaf(n, gam[i], bet[i]));
                p[i] += d;
                q[i] = fmaf(d, n, q[i]);
            }
        });
        const int w = min(c.cols, c.ncols - c0) * V;
        const int second = c.lanes * c.cols * V;
        lane_sums<V>(c, p, q, smem);
        for (int ch = threadIdx.x; ch < w; ch += kGnThreads) {
            part[c0 * V + ch] = smem[ch];
            part[a.C + c0 * V + ch] = smem[second + ch];
        }
        __syncthreads();
    }
}

// The sums of h and h*n over a map, for the groups [g0, g1), from its tiles',
// and the groups' means of gamma*h and gamma*h*n. `lanes` threads per channel
// and sum take every lanes-th tile each, then the lanes in order.
__device__ void join_sums(const GnArgs &a, int b, int map, int g0, int g1, float *smem)
{
    const GnMap m = a.maps[map];
    const int n = (m.rows + a.tr - 1) / a.tr, tid = threadIdx.x, first = g0 * a.Cg, channels = (g1 - g0) * a.Cg;
    const float *part = a.part + (static_cast<int64_t>(b) * a.tiles + m.tile0) * 2 * a.C;
    float *sums = a.sums + (static_cast<int64_t>(b) * a.nmaps + map) * 2 * a.C;
    for (int i0 = 0; i0 < 2 * channels; i0 += kGnThreads) {
        const int w = min(2 * channels - i0, kGnThreads), lanes = kGnThreads / w, lane = tid / w, i = i0 + tid - lane * w;
        const int at = i < channels ? first + i : a.C + first + i - channels;
        float s = 0.f;
        if (lane < lanes)
            for (int t = lane; t < n; t += 16 * lanes) {
                float p[16];
#pragma unroll
                for (int u = 0; u < 16; ++u) p[u] = t + u * lanes < n ? __ldcg(part + static_cast<int64_t>(t + u * lanes) * 2 * a.C + at) : 0.f;
#pragma unroll
                for (int u = 0; u < 16; ++u) s += p[u];
            }
        smem[tid] = s;
        __syncthreads();
        if (tid < w) {
            for (int l = 1; l < lanes; ++l) s += smem[l * w + tid];
            sums[at] = s;
        }
        __syncthreads();
    }
    const int aff = a.affine_scales ? m.scale * a.C : 0;
    const float inv = 1.f / (static_cast<float>(m.rows) * static_cast<float>(a.Cg));
    for (int i = 2 * g0 + tid; i < 2 * g1; i += kGnThreads) {
        const int g = i >> 1, base = (i & 1) * a.C + g * a.Cg;
        float s = 0.f;
        for (int j = 0; j < a.Cg; ++j) s = fmaf(__ldcg(sums + base + j), a.gamma[aff + g * a.Cg + j], s);
        a.group[(static_cast<int64_t>(b) * a.nmaps + map) * a.G * 2 + i] = s * inv;
    }
    __syncthreads();
}

// grad_gamma and grad_beta: the maps' sums in the order (batch item, map), or
// NaN where a map's were left out.
__device__ void param_grads(const GnArgs &a, bool left_out)
{
    const int scales = a.affine_scales ? a.S : 1, maps = a.B * a.nmaps;
    for (int i = threadIdx.x; i < 2 * scales * a.C; i += kGnThreads) {
        const int which = i >= scales * a.C, at = i - which * scales * a.C, s = at / a.C, ch = at - s * a.C;
        const float *p = a.sums + which * a.C + ch;
        float sum = 0.f;
        if (a.affine_scales) {
#pragma unroll 4
            for (int m = s; m < maps; m += a.S) sum += __ldcg(p + static_cast<int64_t>(m) * 2 * a.C);  // map (k, s) is k*S + s
        } else {
#pragma unroll 16
            for (int m = 0; m < maps; ++m) sum += __ldcg(p + static_cast<int64_t>(m) * 2 * a.C);
        }
        (which ? a.grad_gamma : a.grad_beta)[at] = left_out ? NAN : sum;
    }
}

template <typename T, int V, int ACT, typename Ready> __device__ void tile_grad(const GnArgs &a, const Tile &t, Ready ready)
{
    const Cover c = cover<V>(a.C);
    const int64_t bm = static_cast<int64_t>(t.b) * a.nmaps + t.map;
    const float *st = a.stats + bm * a.G * 2, *gr = a.group + bm * a.G * 2;
    const int aff = a.affine_scales ? a.maps[t.map].scale * a.C : 0;
    for (int c0 = 0; c0 < c.ncols; c0 += c.cols) {
        const int col = c0 + c.col;
        const bool on = c.on && col < c.ncols;
        const int64_t at = t.row * a.C + static_cast<int64_t>(on ? col : 0) * V;
        Rows<T, V, true, true, kBwdRows<T, V>> rows;
        rows.begin(c, on, t.rows, a.C, a.x, a.g, at);
        float mean[V], rstd[V], gam[V], bet[V], m1[V], m2[V];  // the last two times rstd
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int ch = (on ? col : 0) * V + i, g = static_cast<int>(a.div_Cg.div(ch));
            const float2 ms = __ldg(reinterpret_cast<const float2 *>(st) + g);
            mean[i] = ms.x;
            rstd[i] = ms.y;
            gam[i] = a.gamma[aff + ch];
            bet[i] = a.beta[aff + ch];
        }
        if (c0 == 0 && !ready()) return tile_nan<T, V>(a, t);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int g = static_cast<int>(a.div_Cg.div((on ? col : 0) * V + i));
            const float2 gm = __ldcg(reinterpret_cast<const float2 *>(gr) + g);
            m1[i] = rstd[i] * gm.x;
            m2[i] = rstd[i] * gm.y;
        }
        rows.each([&](int o, float (&v)[V], const float (&h)[V]) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float n = (v[i] - mean[i]) * rstd[i];
                const float d = h[i] * act_slope<ACT>(fmaf(n, gam[i], bet[i]));
                v[i] = fmaf(gam[i] * rstd[i], d, -m1[i]) - n * m2[i];
            }
            store_row<T, V>(a.y, at + o, v);
        });
    }
}

// ---- tickets ---------------------------------------------------------------

__device__ uint32_t g_gn_gave_up;

__device__ __forceinline__ uint32_t load_acquire(const uint32_t *p)
{
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

enum ItemKind : int { kSums, kOutputs, kJoin };

struct Item {
    int kind, part, id;  // id: a tile's, or (batch item, map)'s
    Tile t;
};

// Tickets before tile p's sums, joins aside: sums and outputs alternate, the
// outputs `lag` tiles behind.
__device__ __forceinline__ int tickets_before(const GnArgs &a, int p) { return p < a.lag ? p : 2 * p - a.lag; }

// The work of ticket i. The joins of a map come right after its last tile's sums.
__device__ __forceinline__ Item item_of(const GnArgs &a, int ticket)
{
    // Maps, over all batch items, whose joins come at or before the ticket.
    int lo = 0, hi = a.B * a.nmaps;
    const auto joins_at = [&](int i) {
        const int b = i / a.nmaps, m = i - b * a.nmaps;
        const int last = b * a.tiles + (m + 1 < a.nmaps ? a.maps[m + 1].tile0 : a.tiles) - 1;
        return tickets_before(a, last) + 1 + i * a.joins;
    };
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (joins_at(mid) <= ticket) lo = mid + 1; else hi = mid;
    }
    Item it;
    it.part = lo > 0 ? ticket - joins_at(lo - 1) : a.joins;
    if (it.part < a.joins) {
        it.kind = kJoin;
        it.id = lo - 1;
        it.t.b = it.id / a.nmaps;
        it.t.map = it.id - it.t.b * a.nmaps;
        return it;
    }
    const int i = ticket - lo * a.joins, j = i - a.lag;
    if (j < 0) {
        it.kind = kSums;
        it.id = i;
    } else if (j < 2 * (a.ntiles - a.lag)) {
        it.kind = j & 1 ? kOutputs : kSums;
        it.id = j & 1 ? j >> 1 : a.lag + (j >> 1);
    } else {
        it.kind = kOutputs;
        it.id = i - a.ntiles;
    }
    it.t = find_tile(a, it.id);
    return it;
}

__device__ __forceinline__ bool wait_for(const uint32_t *counter, uint32_t want, int tries)
{
    for (int i = 0; i < tries; ++i) {
        if (load_acquire(counter) >= want) return true;
        __nanosleep(100);
    }
    atomicOr(&g_gn_gave_up, 1u);
    return false;
}

template <typename T, int V, int ACT, bool BACKWARD>
__global__ void __launch_bounds__(kGnThreads, kGnCtas) gn_kernel(const __grid_constant__ GnArgs a)
{
    extern __shared__ float smem[];
    __shared__ Item item;
    __shared__ uint32_t flag;
    if (threadIdx.x == 0) {
        item = item_of(a, static_cast<int>(atomicAdd(a.tickets, 1u)));
        flag = item.kind != kJoin || wait_for(a.tiles_done + static_cast<int64_t>(item.t.b) * a.nmaps + item.t.map,
                                              (a.maps[item.t.map].rows + a.tr - 1) / a.tr, a.tries);
    }
    __syncthreads();
    const Tile t = item.t;
    const int kind = item.kind;
    const int64_t bm = static_cast<int64_t>(t.b) * a.nmaps + t.map;
    if (kind == kOutputs) {
        const auto ready = [&] {
            if (threadIdx.x == 0) flag = wait_for(a.ready + bm, a.joins, a.tries);
            __syncthreads();
            return flag != 0;
        };
        if (BACKWARD) tile_grad<T, V, ACT>(a, t, ready);
        else tile_apply<T, V, ACT>(a, t, ready);
    } else if (kind == kSums) {
        if (BACKWARD) tile_sums<T, V, ACT>(a, t, item.id, smem);
        else tile_stats<T, V>(a, t, item.id, smem);
        __syncthreads();
        if (threadIdx.x == 0) {
            __threadfence();
            atomicAdd(a.tiles_done + bm, 1u);
        }
    } else {
        const int part = item.part;
        const bool summed = flag;  // if not, no outputs of the map come to be
        if (BACKWARD && summed) join_sums(a, t.b, t.map, part * a.G / a.joins, (part + 1) * a.G / a.joins, smem);
        if (!BACKWARD) summed ? join_stats(a, t.b, t.map, smem) : nan_stats(a, t.b, t.map);
        __syncthreads();
        if (threadIdx.x == 0) {
            __threadfence();
            if (summed) atomicAdd(a.ready + bm, 1u);
            if (BACKWARD) {
                if (!summed) atomicOr(a.left_out, 1u);
                __threadfence();
                flag = atomicAdd(a.all_done, 1u) + 1 == static_cast<uint32_t>(a.B * a.nmaps * a.joins);
                __threadfence();
            }
        }
        __syncthreads();
        if (BACKWARD && flag) param_grads(a, __ldcg(a.left_out) != 0);
    }
}

// Maps of at most kGnSmall bytes: one CTA takes a map from its sums to its
// outputs, without tickets, counters or waits.
template <typename T, int V, int ACT, bool BACKWARD>
__global__ void __launch_bounds__(kGnThreads, kGnCtas) gn_small_kernel(const __grid_constant__ GnArgs a)
{
    extern __shared__ float smem[];
    const Tile t = find_tile(a, blockIdx.x);  // a tile is a whole map
    const auto ready = [] { return true; };
    if (BACKWARD) tile_sums<T, V, ACT>(a, t, blockIdx.x, smem);
    else tile_stats<T, V>(a, t, blockIdx.x, smem);
    __syncthreads();
    if (BACKWARD) join_sums(a, t.b, t.map, 0, a.G, smem);
    else join_stats(a, t.b, t.map, smem);
    __syncthreads();
    if (BACKWARD) tile_grad<T, V, ACT>(a, t, ready);
    else tile_apply<T, V, ACT>(a, t, ready);
    if (BACKWARD && gridDim.x == 1) param_grads(a, false);
}

__global__ void __launch_bounds__(kGnThreads) gn_param_kernel(const __grid_constant__ GnArgs a) { param_grads(a, false); }

struct GnPlan {
    GnArgs a;
    int elem;          // bytes of an element
    bool small;        // every map within kGnSmall bytes
    bool wide;         // rows of whole 16-byte pieces: four channels to an access
    int64_t ntiles;    // B * tiles
    int64_t gaps;      // rows of no map, per batch item
    size_t part, sums, group, counters, total;  // workspace offsets and size
    size_t counter_bytes;
};

size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

da_status gn_plan(const gn_dims *dims, const int32_t *shape, const int32_t *start, bool backward, GnPlan &p)
{
    if (!dims) return fail(DA_ERR_NULL, "dims is NULL");
    const gn_dims d = *dims;
    if (d.batch < 0 || d.num_cams < 0 || d.num_scales < 0) return fail(DA_ERR_SHAPE, "negative size in dims");
    if (d.num_embeds < 1 || d.num_groups < 1 || d.num_embeds % d.num_groups != 0)
        return fail(DA_ERR_SHAPE, "num_embeds (%d) must be a positive multiple of num_groups (%d)", d.num_embeds,
                    d.num_groups);
    if (d.num_embeds > GN_MAX_CHANNELS)
        return fail(DA_ERR_UNSUPPORTED, "num_embeds %d exceeds %d", d.num_embeds, GN_MAX_CHANNELS);
    if (d.feat_dtype != DA_F32 && d.feat_dtype != DA_BF16 && d.feat_dtype != DA_F16)
        return fail(DA_ERR_SHAPE, "unknown feat_dtype %d", d.feat_dtype);
    if (d.act != GN_ACT_NONE && d.act != GN_ACT_RELU && d.act != GN_ACT_SILU)
        return fail(DA_ERR_SHAPE, "unknown act %d", d.act);
    if (!(d.eps > 0.f) || !std::isfinite(d.eps)) return fail(DA_ERR_SHAPE, "eps %g must be positive and finite", d.eps);
    if (d.num_feat_rows < 0 || d.num_feat_rows > DA_MAX_ROWS)
        return fail(DA_ERR_SHAPE, "num_feat_rows %lld outside [0, %d]", static_cast<long long>(d.num_feat_rows),
                    DA_MAX_ROWS);
    const int64_t nmaps = static_cast<int64_t>(d.num_cams) * d.num_scales;
    if (nmaps > DA_MAX_MAPS)
        return fail(DA_ERR_UNSUPPORTED, "num_cams*num_scales = %lld exceeds %d", static_cast<long long>(nmaps), DA_MAX_MAPS);
    if (nmaps > 0 && (!shape || !start)) return fail(DA_ERR_NULL, "spatial_shape / level_start_index is NULL");
    GnArgs &a = p.a;
    int64_t covered = 0;
    for (int i = 0; i < nmaps; ++i) {
        const int32_t H = shape[2 * i], W = shape[2 * i + 1], st = start[i];
        if (H < 1 || W < 1 || H > DA_MAX_MAP_SIDE || W > DA_MAX_MAP_SIDE)
            return fail(DA_ERR_SHAPE, "map %d has shape %d x %d", i, H, W);
        const int64_t n = static_cast<int64_t>(H) * W;
        if (st < 0 || st + n > d.num_feat_rows)
            return fail(DA_ERR_SHAPE, "map %d (start %d, %d x %d) does not fit in %lld feature rows", i, st, H, W,
                        static_cast<long long>(d.num_feat_rows));
        for (int j = 0; j < i; ++j)
            if (st < a.maps[j].start + static_cast<int64_t>(a.maps[j].rows) && a.maps[j].start < st + n)
                return fail(DA_ERR_SHAPE, "maps %d and %d overlap", j, i);
        a.maps[i] = GnMap{static_cast<int32_t>(n), st, 0, static_cast<int32_t>(i % d.num_scales)};
        covered += n;
    }
    // Tiles of about 128 KB forward, 64 KB of each tensor backward, less where
    // that leaves a resident CTA without one, and no fewer than 16 rows. What a
    // CTA does once (ticket, waits, joins of its rows' sums) takes as long as
    // some 20 KB: at 6 x 89760 rows of 256 fp32 channels, forward 378 us with
    // tiles of 32 KB, 260 with 64 and 236 with 128, backward 556, 440 and 428
    // with 32, 64 and 128; but at 1 x 132000 bf16 rows backward 94, 88 and 95.
    const int64_t row_bytes = static_cast<int64_t>(d.num_embeds) * (d.feat_dtype == DA_F32 ? 4 : 2);
    const int64_t by_size = (backward ? 65536 : 131072) / row_bytes, by_count = covered * d.batch / (kGnCtas * 152);
    const int64_t tr = by_size < by_count ? by_size : by_count;
    a.tr = static_cast<int32_t>(tr < 16 ? 16 : tr > 512 ? 512 : tr);
    int64_t tiles = 0, largest = 0, most_rows = 0;
    for (int i = 0; i < nmaps; ++i) most_rows = a.maps[i].rows > most_rows ? a.maps[i].rows : most_rows;
    p.small = most_rows * row_bytes <= kGnSmall;
    if (p.small && most_rows > 0) a.tr = static_cast<int32_t>(most_rows);
    for (int i = 0; i < nmaps; ++i) {
        a.maps[i].tile0 = static_cast<int32_t>(tiles);
        const int64_t n = (a.maps[i].rows + a.tr - 1) / a.tr;
        tiles += n;
        largest = n > largest ? n : largest;
    }
    a.rows = d.num_feat_rows;
    a.B = d.batch;
    a.C = d.num_embeds;
    a.G = d.num_groups;
    a.Cg = a.C / a.G;
    a.div_Cg = FastDiv::make(static_cast<uint32_t>(a.Cg));
    a.nmaps = static_cast<int>(nmaps);
    a.S = d.num_scales;
    a.tiles = static_cast<int32_t>(tiles);
    a.affine_scales = d.affine_scales != 0;
    a.eps = d.eps;
    a.tries = g_gn_tries;
    p.elem = d.feat_dtype == DA_F32 ? 4 : 2;
    p.ntiles = tiles * d.batch;
    p.gaps = d.num_feat_rows - covered;
    if (p.ntiles > INT32_MAX / 4) return fail(DA_ERR_UNSUPPORTED, "too many tiles of %d rows", a.tr);
    a.ntiles = static_cast<int32_t>(p.ntiles);
    // A map's outputs begin two thirds of a resident set of CTAs after its
    // last sums, which are usually joined by then. Twice and three times as
    // many measured within 4 % of it; none at all, 30 % slower.
    const int64_t lag = largest + 2 * 152;
    a.lag = static_cast<int32_t>(lag < p.ntiles ? lag : p.ntiles);
    // A backward join reads 2 C floats of each tile: four CTAs share it.
    a.joins = backward && a.G >= 4 ? 4 : 1;
    const size_t bm = static_cast<size_t>(d.batch) * nmaps;
    size_t at = 0;
    p.part = at;
    at += round256(sizeof(float) * static_cast<size_t>(p.ntiles) * 2 * (backward ? a.C : a.G));
    p.sums = at;
    if (backward) at += round256(sizeof(float) * bm * 2 * a.C);
    p.group = at;
    if (backward) at += round256(sizeof(float) * bm * 2 * a.G);
    p.counters = at;
    p.counter_bytes = p.ntiles > 0 ? sizeof(uint32_t) * (3 + 2 * bm) : 0;
    at += round256(p.counter_bytes);
    p.total = at;
    return DA_OK;
}

da_status gn_buffers(GnPlan &p, const void *x, const void *g, void *y, const float *gamma, const float *beta,
                     const float *stats, void *ws, size_t ws_bytes, bool backward)
{
    GnArgs &a = p.a;
    if (a.rows * a.B > 0 && (!x || !y || (backward && !g))) return fail(DA_ERR_NULL, "a feature tensor is NULL");
    if ((!gamma || !beta) && (a.affine_scales ? a.S : 1) > 0) return fail(DA_ERR_NULL, "gamma or beta is NULL");
    if (p.ntiles > 0 && !stats) return fail(DA_ERR_NULL, "stats is NULL");
    if (!aligned(x, p.elem) || !aligned(y, p.elem) || !aligned(g, p.elem))
        return fail(DA_ERR_ALIGN, "feature tensors must be aligned to their elements");
    if (!aligned(gamma, 4) || !aligned(beta, 4)) return fail(DA_ERR_ALIGN, "gamma and beta must be 4-byte aligned");
    if (!aligned(stats, 8)) return fail(DA_ERR_ALIGN, "stats must be 8-byte aligned");  // a group's pair is one access
    if (p.total > 0) {
        if (!ws || ws_bytes < p.total)
            return fail(DA_ERR_WORKSPACE, "workspace of %zu bytes; %zu are needed", ws ? ws_bytes : size_t{0}, p.total);
        if (!aligned(ws, 256)) return fail(DA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    }
    p.wide = a.C * p.elem % 16 == 0 && aligned(x, 16) && aligned(y, 16) && aligned(g, 16);
    a.x = x;
    a.g = g;
    a.y = y;
    a.gamma = gamma;
    a.beta = beta;
    a.stats = const_cast<float *>(stats);
    char *w = static_cast<char *>(ws);
    a.part = reinterpret_cast<float *>(w + p.part);
    a.sums = reinterpret_cast<float *>(w + p.sums);
    a.group = reinterpret_cast<float *>(w + p.group);
    a.tickets = reinterpret_cast<uint32_t *>(w + p.counters);
    a.all_done = a.tickets + 1;
    a.left_out = a.tickets + 2;
    a.tiles_done = a.tickets + 3;
    a.ready = a.tiles_done + static_cast<int64_t>(a.B) * a.nmaps;
    return DA_OK;
}

// Rows of no map are zeroed by copies from nothing: one memset per stretch
// between maps and batch item.
da_status gn_zero_gaps(const GnPlan &p, cudaStream_t st)
{
    if (p.gaps == 0) return DA_OK;
    const GnArgs &a = p.a;
    const size_t row = static_cast<size_t>(a.C) * p.elem, pitch = row * a.rows;
    int64_t at = 0;
    while (at < a.rows) {
        int64_t next = a.rows, past = a.rows;  // the first map at or after `at`
        for (int i = 0; i < a.nmaps; ++i)
            if (a.maps[i].start >= at && a.maps[i].start < next) {
                next = a.maps[i].start;
                past = next + a.maps[i].rows;
            }
        if (next > at) {
            const cudaError_t e = cudaMemset2DAsync(static_cast<char *>(a.y) + at * row, pitch, 0, (next - at) * row, a.B, st);
            if (e != cudaSuccess) return cuda_fail(e, "zeroing the rows of no map");
        }
        at = past;
    }
    return DA_OK;
}

template <typename T, int V, int ACT, bool BACKWARD> cudaError_t width_launch(const GnPlan &p, cudaStream_t st)
{
    const size_t lanes = 2 * kGnThreads * V + (BACKWARD ? 0 : 2 * p.a.C), smem = sizeof(float) * (lanes < 3 * kGnThreads ? 3 * kGnThreads : lanes);
    if (p.small) {
        gn_small_kernel<T, V, ACT, BACKWARD><<<static_cast<unsigned>(p.ntiles), kGnThreads, smem, st>>>(p.a);
        if (BACKWARD && p.ntiles > 1) gn_param_kernel<<<1, kGnThreads, 0, st>>>(p.a);
        return cudaGetLastError();
    }
    const cudaError_t e = cudaMemsetAsync(p.a.tickets, 0, p.counter_bytes, st);
    if (e != cudaSuccess) return e;
    const unsigned grid = static_cast<unsigned>(2 * p.ntiles + p.a.B * p.a.nmaps * p.a.joins);
    gn_kernel<T, V, ACT, BACKWARD><<<grid, kGnThreads, smem, st>>>(p.a);
    return cudaGetLastError();
}

template <typename T, int ACT, bool BACKWARD> cudaError_t map_launch(const GnPlan &p, cudaStream_t st)
{
    return p.wide ? width_launch<T, 4, ACT, BACKWARD>(p, st) : width_launch<T, 1, ACT, BACKWARD>(p, st);
}

template <typename T> cudaError_t launch_act(const GnPlan &p, int act, bool backward, cudaStream_t st)
{
    if (act == GN_ACT_RELU) return backward ? map_launch<T, GN_ACT_RELU, true>(p, st) : map_launch<T, GN_ACT_RELU, false>(p, st);
    if (act == GN_ACT_SILU) return backward ? map_launch<T, GN_ACT_SILU, true>(p, st) : map_launch<T, GN_ACT_SILU, false>(p, st);
    return backward ? map_launch<T, GN_ACT_NONE, true>(p, st) : map_launch<T, GN_ACT_NONE, false>(p, st);
}

cudaError_t gn_launch(const GnPlan &p, int dtype, int act, bool backward, cudaStream_t st)
{
    if (dtype == DA_F32) return launch_act<float>(p, act, backward, st);
    if (dtype == DA_BF16) return launch_act<__nv_bfloat16>(p, act, backward, st);
    return launch_act<__half>(p, act, backward, st);
}

}  // namespace
}  // namespace da

extern "C" {

da_status gn_workspace_size(const gn_dims *dims, const int32_t *spatial_shape, const int32_t *level_start_index,
                            int32_t backward, size_t *bytes)
{
    if (!bytes) return da::fail(DA_ERR_NULL, "bytes is NULL");
    da::GnPlan p{};
    const da_status st = da::gn_plan(dims, spatial_shape, level_start_index, backward != 0, p);
    if (st != DA_OK) return st;
    *bytes = p.total;
    return DA_OK;
}

da_status gn_forward(const gn_dims *dims, const void *feat, const int32_t *spatial_shape,
                     const int32_t *level_start_index, const float *gamma, const float *beta, void *out, float *stats,
                     void *workspace, size_t workspace_bytes, da_stream_t stream)
{
    da::GnPlan p{};
    da_status st = da::gn_plan(dims, spatial_shape, level_start_index, false, p);
    if (st != DA_OK) return st;
    st = da::gn_buffers(p, feat, nullptr, out, gamma, beta, stats, workspace, workspace_bytes, false);
    if (st != DA_OK) return st;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if ((st = da::gn_zero_gaps(p, cs)) != DA_OK || p.ntiles == 0) return st;
    const cudaError_t e = da::gn_launch(p, dims->feat_dtype, dims->act, false, cs);
    return e == cudaSuccess ? DA_OK : da::cuda_fail(e, "group norm launch");
}

da_status gn_backward(const gn_dims *dims, const void *feat, const int32_t *spatial_shape,
                      const int32_t *level_start_index, const float *gamma, const float *beta, const float *stats,
                      const void *grad_out, void *grad_feat, float *grad_gamma, float *grad_beta, void *workspace,
                      size_t workspace_bytes, da_stream_t stream)
{
    da::GnPlan p{};
    da_status st = da::gn_plan(dims, spatial_shape, level_start_index, true, p);
    if (st != DA_OK) return st;
    st = da::gn_buffers(p, feat, grad_out, grad_feat, gamma, beta, stats, workspace, workspace_bytes, true);
    if (st != DA_OK) return st;
    const int params = (p.a.affine_scales ? p.a.S : 1) * p.a.C;
    if (params > 0 && (!grad_gamma || !grad_beta)) return da::fail(DA_ERR_NULL, "grad_gamma or grad_beta is NULL");
    if (!da::aligned(grad_gamma, 4) || !da::aligned(grad_beta, 4))
        return da::fail(DA_ERR_ALIGN, "grad_gamma and grad_beta must be 4-byte aligned");
    p.a.grad_gamma = grad_gamma;
    p.a.grad_beta = grad_beta;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if ((st = da::gn_zero_gaps(p, cs)) != DA_OK) return st;
    if (p.ntiles > 0) {
        const cudaError_t e = da::gn_launch(p, dims->feat_dtype, dims->act, true, cs);
        if (e != cudaSuccess) return da::cuda_fail(e, "group norm backward launch");
    }
    if (p.ntiles == 0 && params > 0) {  // sums over nothing
        cudaError_t e = cudaMemsetAsync(grad_gamma, 0, sizeof(float) * params, cs);
        if (e == cudaSuccess) e = cudaMemsetAsync(grad_beta, 0, sizeof(float) * params, cs);
        if (e != cudaSuccess) return da::cuda_fail(e, "group norm parameter gradients");
    }
    return DA_OK;
}

int32_t da_gn_wait_tries(int32_t tries) { return tries < 0 ? da::g_gn_tries.load() : da::g_gn_tries.exchange(tries); }

da_status gn_device_status(uint32_t *gave_up, da_stream_t stream)
{
    if (!gave_up) return da::fail(DA_ERR_NULL, "gave_up is NULL");
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    void *word = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&word, da::g_gn_gave_up);
    if (e == cudaSuccess) e = cudaMemcpyAsync(gave_up, word, sizeof *gave_up, cudaMemcpyDeviceToHost, cs);
    if (e == cudaSuccess) e = cudaMemsetAsync(word, 0, sizeof *gave_up, cs);
    if (e == cudaSuccess) e = cudaStreamSynchronize(cs);
    return e == cudaSuccess ? DA_OK : da::cuda_fail(e, "status word");
}

}  // extern "C"
