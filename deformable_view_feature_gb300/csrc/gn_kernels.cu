// Group norm with an activation over packed channels-last maps (include/gn.h).
//
// A map is cut into tiles of `tr` rows. One pass takes every tile's sums, one
// CTA per (batch item, map) joins them in the order of the tiles, and a second
// pass over the tiles writes the outputs. A CTA's threads form a grid of
// 16-byte columns x rows of its tile, so every access is a full row segment
// and a thread keeps its channels' parameters in registers.
//
// Forward statistics: a tile sums x - p and (x - p)^2 per channel, p being
// the tile's first row, and turns them into a mean and a sum of squared
// deviations per group; tiles are then joined by
//   M2 = sum M2_t + sum n_t (mean_t - mean)^2.
// No sum of squares about zero occurs, so a mean far larger than the spread
// costs no digits.
#include <cmath>
#include <cuda_bf16.h>

#include "da_internal.cuh"
#include "gn.h"

namespace da {
namespace {

constexpr int kGnThreads = 256;

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
    int64_t rows;        // per batch item
    int32_t B, C, G, Cg, nmaps, S, K, tiles, tr, affine_scales;
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

// V consecutive channels: 16 bytes, or one element where rows are not
// multiples of 16 bytes.
template <typename T, int V> struct alignas(sizeof(T) * V) Pack {
    T v[V];
};

template <typename T, int V> __device__ __forceinline__ void load_row(const void *base, int64_t at, float (&f)[V])
{
    const Pack<T, V> p = *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(base) + at);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = to_f(p.v[i]);
}

template <typename T, int V> __device__ __forceinline__ void store_row(void *base, int64_t at, const float (&f)[V])
{
    Pack<T, V> p;
#pragma unroll
    for (int i = 0; i < V; ++i) p.v[i] = from_f<T>(f[i]);
    *reinterpret_cast<Pack<T, V> *>(static_cast<T *>(base) + at) = p;
}

// act(z), and act'(z) for the backward pass.
template <int ACT> __device__ __forceinline__ float act_of(float z)
{
    if (ACT == GN_ACT_RELU) return z < 0.f ? 0.f : z;  // NaN stays NaN
    if (ACT == GN_ACT_SILU) return __fdividef(z, 1.f + __expf(-z));
    return z;
}
template <int ACT> __device__ __forceinline__ float act_slope(float z)
{
    if (ACT == GN_ACT_RELU) return z > 0.f ? 1.f : 0.f;
    if (ACT == GN_ACT_SILU) {
        const float s = __fdividef(1.f, 1.f + __expf(-z));
        return s * (1.f + z * (1.f - s));
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
    const float inv = 1.f / static_cast<float>(t.rows);
    for (int c0 = 0; c0 < c.ncols; c0 += c.cols) {
        const int col = c0 + c.col;
        const bool on = c.on && col < c.ncols;
        float p[V], s[V], q[V];
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = s[i] = q[i] = 0.f;
        if (on) {
            const int64_t at = t.row * a.C + static_cast<int64_t>(col) * V;
            load_row<T, V>(a.x, at, p);
#pragma unroll 4
            for (int r = c.lane; r < t.rows; r += c.lanes) {
                float v[V];
                load_row<T, V>(a.x, at + static_cast<int64_t>(r) * a.C, v);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float d = v[i] - p[i];
                    s[i] += d;
                    q[i] = fmaf(d, d, q[i]);
                }
            }
        }
        const int w = min(c.cols, c.ncols - c0) * V;
        const int second = c.lanes * c.cols * V;
        lane_sums<V>(c, s, q, scratch);
        for (int ch = threadIdx.x; ch < w; ch += kGnThreads) {
            const float sum = scratch[ch], sq = scratch[second + ch];
            const float piv = to_f(static_cast<const T *>(a.x)[t.row * a.C + static_cast<int64_t>(c0) * V + ch]);
            mean_c[c0 * V + ch] = piv + sum * inv;
            m2_c[c0 * V + ch] = fmaxf(sq - sum * sum * inv, 0.f);
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

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One warp per group: joins the tiles' means and squared deviations.
__device__ void join_stats(const GnArgs &a, int b, int map)
{
    const GnMap m = a.maps[map];
    const int n = (m.rows + a.tr - 1) / a.tr;
    const int lane = threadIdx.x & 31;
    const float *part = a.part + (static_cast<int64_t>(b) * a.tiles + m.tile0) * a.G * 2;
    const float inv_rows = 1.f / static_cast<float>(m.rows);
    for (int g = threadIdx.x >> 5; g < a.G; g += kGnThreads / 32) {
        // The mean is taken about the first tile's, the deviations about it.
        const float base = part[g * 2];
        float s = 0.f;
        for (int t = lane; t < n; t += 32)
            s += (part[(static_cast<int64_t>(t) * a.G + g) * 2] - base) * static_cast<float>(min(a.tr, m.rows - t * a.tr));
        const float mean = base + warp_sum(s) * inv_rows;
        float q = 0.f;
        for (int t = lane; t < n; t += 32) {
            const float *p = part + (static_cast<int64_t>(t) * a.G + g) * 2;
            const float d = p[0] - mean;
            q += p[1] + d * d * static_cast<float>(min(a.tr, m.rows - t * a.tr)) * static_cast<float>(a.Cg);
        }
        q = warp_sum(q);
        if (lane == 0) {
            float *o = a.stats + ((static_cast<int64_t>(b) * a.nmaps + map) * a.G + g) * 2;
            o[0] = mean;
            o[1] = 1.f / sqrtf(q * inv_rows / static_cast<float>(a.Cg) + a.eps);
        }
    }
}

template <typename T, int V, int ACT> __device__ void tile_apply(const GnArgs &a, const Tile &t)
{
    const Cover c = cover<V>(a.C);
    if (!c.on) return;
    const float *st = a.stats + (static_cast<int64_t>(t.b) * a.nmaps + t.map) * a.G * 2;
    const int aff = a.affine_scales ? a.maps[t.map].scale * a.C : 0;
    for (int col = c.col; col < c.ncols; col += c.cols) {
        float mean[V], mul[V], add[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int ch = col * V + i, g = ch / a.Cg;
            mean[i] = st[g * 2];
            mul[i] = st[g * 2 + 1] * a.gamma[aff + ch];
            add[i] = a.beta[aff + ch];
        }
        const int64_t at = t.row * a.C + static_cast<int64_t>(col) * V;
#pragma unroll 4
        for (int r = c.lane; r < t.rows; r += c.lanes) {
            float v[V];
            load_row<T, V>(a.x, at + static_cast<int64_t>(r) * a.C, v);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = act_of<ACT>(fmaf(v[i] - mean[i], mul[i], add[i]));
            store_row<T, V>(a.y, at + static_cast<int64_t>(r) * a.C, v);
        }
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
        float p[V], q[V];
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = q[i] = 0.f;
        if (c.on && col < c.ncols) {
            float mean[V], rstd[V], gam[V], bet[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int ch = col * V + i, g = ch / a.Cg;
                mean[i] = st[g * 2];
                rstd[i] = st[g * 2 + 1];
                gam[i] = a.gamma[aff + ch];
                bet[i] = a.beta[aff + ch];
            }
            const int64_t at = t.row * a.C + static_cast<int64_t>(col) * V;
#pragma unroll 4
            for (int r = c.lane; r < t.rows; r += c.lanes) {
                float v[V], h[V];
                load_row<T, V>(a.x, at + static_cast<int64_t>(r) * a.C, v);
                load_row<T, V>(a.g, at + static_cast<int64_t>(r) * a.C, h);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float n = (v[i] - mean[i]) * rstd[i];
                    const float d = h[i] * act_slope<ACT>(fmaf(n, gam[i], bet[i]));
                    p[i] += d;
                    q[i] = fmaf(d, n, q[i]);
                }
            }
        }
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

// Joins the tiles of (b, map): the channels' sums and the groups' means.
__device__ void join_sums(const GnArgs &a, int b, int map, float *smem)
{
    const GnMap m = a.maps[map];
    const int n = (m.rows + a.tr - 1) / a.tr;
    const float *part = a.part + (static_cast<int64_t>(b) * a.tiles + m.tile0) * 2 * a.C;
    float *sums = a.sums + (static_cast<int64_t>(b) * a.nmaps + map) * 2 * a.C;
    const int aff = a.affine_scales ? m.scale * a.C : 0;
    for (int i = threadIdx.x; i < 2 * a.C; i += kGnThreads) {
        float s = 0.f;
#pragma unroll 8
        for (int t = 0; t < n; ++t) s += part[static_cast<int64_t>(t) * 2 * a.C + i];
        sums[i] = s;
        smem[i] = s * a.gamma[aff + (i >= a.C ? i - a.C : i)];
    }
    __syncthreads();
    const float inv = 1.f / (static_cast<float>(m.rows) * static_cast<float>(a.Cg));
    for (int i = threadIdx.x; i < 2 * a.G; i += kGnThreads) {
        const int g = i >> 1, base = (i & 1) * a.C + g * a.Cg;
        float s = 0.f;
        for (int j = 0; j < a.Cg; ++j) s += smem[base + j];
        a.group[(static_cast<int64_t>(b) * a.nmaps + map) * a.G * 2 + i] = s * inv;
    }
}

template <typename T, int V, int ACT> __device__ void tile_grad(const GnArgs &a, const Tile &t)
{
    const Cover c = cover<V>(a.C);
    if (!c.on) return;
    const int64_t bm = static_cast<int64_t>(t.b) * a.nmaps + t.map;
    const float *st = a.stats + bm * a.G * 2, *gr = a.group + bm * a.G * 2;
    const int aff = a.affine_scales ? a.maps[t.map].scale * a.C : 0;
    for (int col = c.col; col < c.ncols; col += c.cols) {
        float mean[V], rstd[V], gam[V], bet[V], m1[V], m2[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int ch = col * V + i, g = ch / a.Cg;
            mean[i] = st[g * 2];
            rstd[i] = st[g * 2 + 1];
            m1[i] = gr[g * 2];
            m2[i] = gr[g * 2 + 1];
            gam[i] = a.gamma[aff + ch];
            bet[i] = a.beta[aff + ch];
        }
        const int64_t at = t.row * a.C + static_cast<int64_t>(col) * V;
#pragma unroll 2
        for (int r = c.lane; r < t.rows; r += c.lanes) {
            float v[V], h[V];
            load_row<T, V>(a.x, at + static_cast<int64_t>(r) * a.C, v);
            load_row<T, V>(a.g, at + static_cast<int64_t>(r) * a.C, h);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float n = (v[i] - mean[i]) * rstd[i];
                const float d = h[i] * act_slope<ACT>(fmaf(n, gam[i], bet[i]));
                v[i] = rstd[i] * (fmaf(gam[i], d, -m1[i]) - n * m2[i]);
            }
            store_row<T, V>(a.y, at + static_cast<int64_t>(r) * a.C, v);
        }
    }
}

// ---- kernels ---------------------------------------------------------------

template <typename T, int V> __global__ void __launch_bounds__(kGnThreads) gn_stats_kernel(const __grid_constant__ GnArgs a)
{
    extern __shared__ float smem[];
    tile_stats<T, V>(a, find_tile(a, blockIdx.x), blockIdx.x, smem);
}

__global__ void __launch_bounds__(kGnThreads) gn_join_stats_kernel(const __grid_constant__ GnArgs a)
{
    join_stats(a, blockIdx.x / a.nmaps, blockIdx.x % a.nmaps);
}

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kGnThreads) gn_apply_kernel(const __grid_constant__ GnArgs a)
{
    tile_apply<T, V, ACT>(a, find_tile(a, blockIdx.x));
}

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kGnThreads) gn_sums_kernel(const __grid_constant__ GnArgs a)
{
    extern __shared__ float smem[];
    tile_sums<T, V, ACT>(a, find_tile(a, blockIdx.x), blockIdx.x, smem);
}

__global__ void __launch_bounds__(kGnThreads) gn_join_sums_kernel(const __grid_constant__ GnArgs a)
{
    extern __shared__ float smem[];
    join_sums(a, blockIdx.x / a.nmaps, blockIdx.x % a.nmaps, smem);
}

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kGnThreads) gn_grad_kernel(const __grid_constant__ GnArgs a)
{
    tile_grad<T, V, ACT>(a, find_tile(a, blockIdx.x));
}

// grad_gamma and grad_beta: the maps' sums in the order (batch item, map).
__global__ void __launch_bounds__(kGnThreads) gn_param_kernel(const __grid_constant__ GnArgs a)
{
    const int scales = a.affine_scales ? a.S : 1;
    const int i = blockIdx.x * kGnThreads + threadIdx.x;
    if (i >= scales * a.C) return;
    const int s = i / a.C, ch = i - s * a.C;
    float sg = 0.f, sb = 0.f;
    for (int b = 0; b < a.B; ++b)
        for (int m = 0; m < a.nmaps; ++m) {
            if (a.affine_scales && a.maps[m].scale != s) continue;
            const float *p = a.sums + (static_cast<int64_t>(b) * a.nmaps + m) * 2 * a.C + ch;
            sb += p[0];
            sg += p[a.C];
        }
    a.grad_gamma[i] = sg;
    a.grad_beta[i] = sb;
}

struct GnPlan {
    GnArgs a;
    int elem, vec;     // bytes of an element, elements per access
    int64_t ntiles;    // B * tiles
    int64_t gaps;      // rows of no map, per batch item
    size_t part, sums, group, total;  // workspace offsets and size
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
    // 64-row tiles. Fewer rows per tile only add sums to join; more leave
    // the smallest maps of a pyramid to too few CTAs.
    a.tr = 64;
    int64_t tiles = 0;
    for (int i = 0; i < nmaps; ++i) {
        a.maps[i].tile0 = static_cast<int32_t>(tiles);
        tiles += (a.maps[i].rows + a.tr - 1) / a.tr;
    }
    a.rows = d.num_feat_rows;
    a.B = d.batch;
    a.C = d.num_embeds;
    a.G = d.num_groups;
    a.Cg = a.C / a.G;
    a.nmaps = static_cast<int>(nmaps);
    a.S = d.num_scales;
    a.K = d.num_cams;
    a.tiles = static_cast<int32_t>(tiles);
    a.affine_scales = d.affine_scales != 0;
    a.eps = d.eps;
    p.elem = d.feat_dtype == DA_F32 ? 4 : 2;
    p.ntiles = tiles * d.batch;
    p.gaps = d.num_feat_rows - covered;
    if (p.ntiles > INT32_MAX) return fail(DA_ERR_UNSUPPORTED, "more than 2^31 tiles of %d rows", a.tr);
    const size_t bm = static_cast<size_t>(d.batch) * nmaps;
    size_t at = 0;
    p.part = at;
    at += round256(sizeof(float) * static_cast<size_t>(p.ntiles) * 2 * (backward ? a.C : a.G));
    p.sums = at;
    if (backward) at += round256(sizeof(float) * bm * 2 * a.C);
    p.group = at;
    if (backward) at += round256(sizeof(float) * bm * 2 * a.G);
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
    if (!aligned(gamma, 4) || !aligned(beta, 4) || !aligned(stats, 4))
        return fail(DA_ERR_ALIGN, "gamma, beta and stats must be 4-byte aligned");
    if (p.total > 0) {
        if (!ws || ws_bytes < p.total)
            return fail(DA_ERR_WORKSPACE, "workspace of %zu bytes; %zu are needed", ws ? ws_bytes : size_t{0}, p.total);
        if (!aligned(ws, 256)) return fail(DA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    }
    const bool wide = a.C * p.elem % 16 == 0 && aligned(x, 16) && aligned(y, 16) && aligned(g, 16);
    p.vec = wide ? 16 / p.elem : 1;
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

template <typename T, int V, int ACT> cudaError_t forward_launch(const GnPlan &p, cudaStream_t st)
{
    const unsigned n = static_cast<unsigned>(p.ntiles);
    const size_t smem = sizeof(float) * (2 * kGnThreads * V + 2 * p.a.C);
    gn_stats_kernel<T, V><<<n, kGnThreads, smem, st>>>(p.a);
    gn_join_stats_kernel<<<p.a.B * p.a.nmaps, kGnThreads, 0, st>>>(p.a);
    gn_apply_kernel<T, V, ACT><<<n, kGnThreads, 0, st>>>(p.a);
    return cudaGetLastError();
}

template <typename T, int V, int ACT> cudaError_t backward_launch(const GnPlan &p, cudaStream_t st)
{
    const unsigned n = static_cast<unsigned>(p.ntiles);
    gn_sums_kernel<T, V, ACT><<<n, kGnThreads, sizeof(float) * 2 * kGnThreads * V, st>>>(p.a);
    gn_join_sums_kernel<<<p.a.B * p.a.nmaps, kGnThreads, sizeof(float) * 2 * p.a.C, st>>>(p.a);
    gn_grad_kernel<T, V, ACT><<<n, kGnThreads, 0, st>>>(p.a);
    return cudaGetLastError();
}

template <typename T, int V> cudaError_t launch_act(const GnPlan &p, int act, bool backward, cudaStream_t st)
{
    if (act == GN_ACT_RELU) return backward ? backward_launch<T, V, GN_ACT_RELU>(p, st) : forward_launch<T, V, GN_ACT_RELU>(p, st);
    if (act == GN_ACT_SILU) return backward ? backward_launch<T, V, GN_ACT_SILU>(p, st) : forward_launch<T, V, GN_ACT_SILU>(p, st);
    return backward ? backward_launch<T, V, GN_ACT_NONE>(p, st) : forward_launch<T, V, GN_ACT_NONE>(p, st);
}

cudaError_t gn_launch(const GnPlan &p, int dtype, int act, bool backward, cudaStream_t st)
{
    const bool wide = p.vec > 1;
    switch (dtype) {
    case DA_F32: return wide ? launch_act<float, 4>(p, act, backward, st) : launch_act<float, 1>(p, act, backward, st);
    case DA_BF16:
        return wide ? launch_act<__nv_bfloat16, 8>(p, act, backward, st) : launch_act<__nv_bfloat16, 1>(p, act, backward, st);
    default: return wide ? launch_act<__half, 8>(p, act, backward, st) : launch_act<__half, 1>(p, act, backward, st);
    }
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
    if (params > 0) {
        da::gn_param_kernel<<<(params + da::kGnThreads - 1) / da::kGnThreads, da::kGnThreads, 0, cs>>>(p.a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return da::cuda_fail(e, "group norm parameter gradients");
    }
    return DA_OK;
}

}  // extern "C"
