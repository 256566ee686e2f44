// What the general kernels of the differential attention (dattn_general.cu) and
// of its form over a paged cache (paged_general.cu) share: tiles on the fp32
// units and the forward kernel. Nothing here is exported.
#pragma once

#include "dattn_internal.cuh"

namespace da {
namespace {

constexpr int kThreadsG = 256;

__device__ __forceinline__ float4 lds4(const float *p) { return *reinterpret_cast<const float4 *>(p); }

// acc[i][j] = sum_d A[ty + 16 i][d] * B[tx + 16 j][d]
template <int M, int N, int DP>
__device__ __forceinline__ void scores(const float *A, const float *B, int ty, int tx, float (&acc)[M][N])
{
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) acc[i][j] = 0.f;
#pragma unroll 4
    for (int d = 0; d < DP; d += 4) {
        float4 x[M], y[N];
#pragma unroll
        for (int i = 0; i < M; ++i) x[i] = lds4(A + (ty + 16 * i) * (DP + 4) + d);
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] = lds4(B + (tx + 16 * j) * (DP + 4) + d);
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                acc[i][j] = fmaf(x[i].x, y[j].x, acc[i][j]);
                acc[i][j] = fmaf(x[i].y, y[j].y, acc[i][j]);
                acc[i][j] = fmaf(x[i].z, y[j].z, acc[i][j]);
                acc[i][j] = fmaf(x[i].w, y[j].w, acc[i][j]);
            }
    }
}

__device__ __forceinline__ void fma4(float4 &a, float s, const float4 &v)
{
    a.x = fmaf(s, v.x, a.x);
    a.y = fmaf(s, v.y, a.y);
    a.z = fmaf(s, v.z, a.z);
    a.w = fmaf(s, v.w, a.w);
}

// acc[i][c] += sum_n P[ty + 16 i][n] * V[n][4 tx + 64 c ..]; columns past W
// (a padded width below 64) are not touched.
template <int M, int NT, int W, int NC>
__device__ __forceinline__ void products(const float *P, const float *V, int ty, int tx, float4 (&acc)[M][NC])
{
    if (W < 64 && 4 * tx >= W) return;
#pragma unroll 2
    for (int n = 0; n < NT; n += 4) {
        float4 p[M];
#pragma unroll
        for (int i = 0; i < M; ++i) p[i] = lds4(P + (ty + 16 * i) * (NT + 4) + n);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const float *v = V + n * (W + 4) + 4 * tx + 64 * c;
            const float4 v0 = lds4(v), v1 = lds4(v + (W + 4)), v2 = lds4(v + 2 * (W + 4)), v3 = lds4(v + 3 * (W + 4));
#pragma unroll
            for (int i = 0; i < M; ++i) {
                fma4(acc[i][c], p[i].x, v0);
                fma4(acc[i][c], p[i].y, v1);
                fma4(acc[i][c], p[i].z, v2);
                fma4(acc[i][c], p[i].w, v3);
            }
        }
    }
}

// Sum or maximum over the 16 threads of a row.
__device__ __forceinline__ float row_sum(float v)
{
#pragma unroll
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float row_max(float v)
{
#pragma unroll
    for (int o = 8; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// The bias table of the CTA's G heads, times log2(e), and the bucket map.
struct BiasTable {
    float *table;     // [nb][G]
    uint16_t *map;    // [2 reach + 1]
};

__device__ __forceinline__ size_t bias_floats(int nb, int G, int reach)
{
    return nb ? nb * G + (2 * reach + 2) / 2 + 2 : 0;
}

__device__ void load_bias(const DattnArgs &a, int n, const BiasTable &t)
{
    for (int i = threadIdx.x; i < a.nb * a.G; i += kThreadsG)
        t.table[i] = a.table[(i / a.G) * a.H + n * a.G + i % a.G] * kLog2e;
    for (int i = threadIdx.x; i < 2 * a.reach + 1 && a.nb; i += kThreadsG)
        t.map[i] = static_cast<uint16_t>(min(max(a.bmap[i], 0), a.nb - 1));
}

__device__ __forceinline__ int bucket_of(const DattnArgs &a, const BiasTable &t, int rel)
{
    return t.map[min(max(rel, -a.reach), a.reach) + a.reach];
}

// The bias of a pair, times log2(e); -infinity where the query does not see
// the key. The same for both maps.
__device__ __forceinline__ float bias_of(const DattnArgs &a, const BiasTable &t, int seen, int rel, int g)
{
    const float b = a.nb ? t.table[bucket_of(a, t, rel) * a.G + g] : 0.f;
    return seen && !(a.causal && rel > 0) ? b : -INFINITY;
}

// Per-row data of a tile of rows.
struct RowInfo {
    int pos, g;  // position, head within the key head's group
    int l;       // query, or -1 past the end
};

__device__ __forceinline__ RowInfo row_info(const DattnArgs &a, int b, int len, int r)
{
    RowInfo i{0, 0, -1};
    if (r < a.rows) {
        i.l = static_cast<int>(a.div_G.div(r));
        i.g = r - i.l * a.G;
        i.pos = a.pos_q ? a.pos_q[static_cast<int64_t>(b) * a.Lq + i.l] : len - a.Lq + i.l;
    }
    return i;
}

// Four channels d .. d + 3 of a row, zeros past the width. `wide`: fp32 rows
// that 16-byte loads may read, whose width is a multiple of four.
template <typename T> __device__ __forceinline__ float4 load4(const T *row, int d, int width, bool wide)
{
    if constexpr (sizeof(T) == 4)
        if (wide) return d < width ? *reinterpret_cast<const float4 *>(row + d) : make_float4(0.f, 0.f, 0.f, 0.f);
    return make_float4(d < width ? dattn_float(row[d]) : 0.f, d + 1 < width ? dattn_float(row[d + 1]) : 0.f,
                       d + 2 < width ? dattn_float(row[d + 2]) : 0.f, d + 3 < width ? dattn_float(row[d + 3]) : 0.f);
}

// Tile of rows of a tensor with two maps (or one) to shared memory as fp32;
// channels past the width and rows without a query are zeros.
template <typename T, int W>
__device__ void load_rows(const DattnArgs &a, const void *base, int64_t at, int64_t sl, int64_t sh, int n, int r0,
                          int count, int width, float *dst)
{
#pragma unroll 4
    for (int i = threadIdx.x; i < count * (W / 4); i += kThreadsG) {
        const int row = i / (W / 4), d = (i - row * (W / 4)) * 4, r = r0 + row;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < a.rows) {
            const int l = static_cast<int>(a.div_G.div(r)), g = r - l * a.G;
            v = load4(static_cast<const T *>(base) + at + l * sl + static_cast<int64_t>(n * a.G + g) * sh, d, width, a.wide);
        }
        *reinterpret_cast<float4 *>(dst + row * (W + 4) + d) = v;
    }
}

// Tile of keys or values; keys that are not to be used are zeros.
template <typename T, int W>
__device__ void load_keys(const DattnArgs &a, const void *base, int64_t at, int64_t sl, int j0, int count, int width,
                          const int *seen, float *dst)
{
#pragma unroll 4
    for (int i = threadIdx.x; i < count * (W / 4); i += kThreadsG) {
        const int row = i / (W / 4), d = (i - row * (W / 4)) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (seen[row]) v = load4(static_cast<const T *>(base) + at + (j0 + row) * sl, d, width, a.wide);
        *reinterpret_cast<float4 *>(dst + row * (W + 4) + d) = v;
    }
}

// The same from a paged cache, whose rows lie at `at` [count].
template <typename T, int W>
__device__ void load_paged(const DattnArgs &a, const void *base, int64_t first, int64_t s_page, int64_t s_place, int count,
                           int width, const int *seen, const int2 *at, float *dst)
{
#pragma unroll 4
    for (int i = threadIdx.x; i < count * (W / 4); i += kThreadsG) {
        const int row = i / (W / 4), d = (i - row * (W / 4)) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (seen[row]) v = load4(static_cast<const T *>(base) + first + at[row].x * s_page + at[row].y * s_place, d, width, a.wide);
        *reinterpret_cast<float4 *>(dst + row * (W + 4) + d) = v;
    }
}

// The same in two halves, so that a step's rows are on their way while the one
// before is worked on: N pieces of a thread's own, asked for and then stored.
template <typename T, int W, int N>
__device__ __forceinline__ void ask_paged(const DattnArgs &a, const void *base, int64_t first, int64_t s_page, int64_t s_place,
                                          int width, const int *seen, const int2 *at, float4 (&r)[N])
{
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const int i = threadIdx.x + u * kThreadsG, row = i / (W / 4), d = (i - row * (W / 4)) * 4;
        r[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (seen[row]) r[u] = load4(static_cast<const T *>(base) + first + at[row].x * s_page + at[row].y * s_place, d, width, a.wide);
    }
}
template <int W, int N> __device__ __forceinline__ void put_paged(const float4 (&r)[N], float *dst)
{
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const int i = threadIdx.x + u * kThreadsG, row = i / (W / 4), d = (i - row * (W / 4)) * 4;
        *reinterpret_cast<float4 *>(dst + row * (W + 4) + d) = r[u];
    }
}

struct PagedKey {
    int2 at;
    int seen, pos;
};

// Position, use and place of key j of a paged cache.
__device__ __forceinline__ PagedKey paged_key(const DattnArgs &a, int b, int end, int j)
{
    PagedKey k{make_int2(-1, 0), 0, j};
    if (j < end) {
        const int64_t of = static_cast<int64_t>(b) * a.Lk + j;
        k.at.x = paged_page(a, b, j, k.at.y);
        k.seen = k.at.x >= 0 && (!a.mask || a.mask[of]);
        if (a.pos_k) k.pos = a.pos_k[of];
    }
    return k;
}

// Positions, use and places of the keys j0 .. of a paged cache.
__device__ __forceinline__ void load_paged_info(const DattnArgs &a, int b, int end, int j0, int count, int *pos, int *seen, int2 *at)
{
    for (int i = threadIdx.x; i < count; i += kThreadsG) {
        const PagedKey k = paged_key(a, b, end, j0 + i);
        at[i] = k.at;
        seen[i] = k.seen;
        pos[i] = k.pos;
    }
}

// Whether new token l sees key j, below the sequence's length, by the tree;
// `old`: the keys before the new ones.
__device__ __forceinline__ bool tree_sees(const DattnArgs &a, int b, int l, int j, int old)
{
    return j < old || a.pg.tree[(static_cast<int64_t>(b) * a.Lq + l) * a.Lq + j - old];
}

// Positions and use of the keys j0 .. j0 + count - 1.
__device__ __forceinline__ void load_key_info(const DattnArgs &a, int b, int end, int j0, int count, int *pos, int *seen)
{
    for (int i = threadIdx.x; i < count; i += kThreadsG) {
        const int j = j0 + i;
        const bool in = j < end;
        const int64_t at = static_cast<int64_t>(b) * a.Lk + j;
        seen[i] = in && (!a.mask || a.mask[at]);
        pos[i] = in && a.pos_k ? a.pos_k[at] : j;
    }
}

// ---- forward ---------------------------------------------------------------

template <typename T, int DP, int QT> struct FwdTile {
    static constexpr int KT = DP <= 64 ? 64 : 32;
    static constexpr int WV = 2 * DP;
    static constexpr int M = QT / 16, N = KT / 16, NC = WV / 64;
    static constexpr int q = 0, k = q + 2 * QT * (DP + 4), v = k + 2 * KT * (DP + 4), p = v + KT * (WV + 4),
                         info = p + 2 * QT * (KT + 4), floats = info + 2 * KT;
};

template <typename T, int DP, int QT, bool PAGED>
__global__ void __launch_bounds__(kThreadsG, DP == 32 || (DP == 64 && QT == 16) ? 2 : 1) dattn_fwd_kernel(const __grid_constant__ DattnArgs a)
{
    using F = FwdTile<T, DP, QT>;
    constexpr int M = F::M, N = F::N, NC = F::NC, KT = F::KT;
    extern __shared__ float sm[];
    float *sq = sm + F::q, *sk = sm + F::k, *sv = sm + F::v, *sp = sm + F::p;
    int *kpos = reinterpret_cast<int *>(sm + F::info), *kseen = kpos + KT;
    const BiasTable bt{sm + F::floats, reinterpret_cast<uint16_t *>(sm + F::floats + a.nb * a.G)};
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int tile = blockIdx.x / a.splits, split = blockIdx.x - tile * a.splits;
    const int n = blockIdx.y, b = blockIdx.z, r0 = tile * QT;
    const int len = dattn_length(a, b);
    // Paged: pages and places of the keys, and their infos, of up to three steps.
    // Their rows are fetched into registers a step ahead, values while scores are
    // formed, where registers allow it (widths up to 64): 60 rows over 2,100 keys
    // six times in fp32 take 60 us, 67 without; 300 tokens of 8 heads over 3,000
    // keys four times 523 us, 755 without. The fp32 units and the reads of shared
    // memory that feed them bound it.
    constexpr bool AHEAD = PAGED && DP <= 64;
    constexpr int NKA = KT * DP / 4 / kThreadsG, NVA = KT * F::WV / 4 / kThreadsG;
    __shared__ int2 at[PAGED ? 3 * KT : 1];
    __shared__ int infos[AHEAD ? 6 * KT : 1];
    float4 ak[2][AHEAD ? NKA : 1], av[AHEAD ? NVA : 1];
    PagedKey ahead{};
    int step = 0;
    const int count = PAGED ? paged_count(a, b) : a.Lq, old = len - count;  // queries, keys before them

    load_bias(a, n, bt);
    for (int m = 0; m < 2; ++m)
        load_rows<T, DP>(a, a.q, b * a.qs[0] + m * a.qs[3], a.qs[1], a.qs[2], n, r0, QT, a.D, sq + m * QT * (DP + 4));
    RowInfo ri[M];
    float mx[2][M], sum[2][M];
    float4 acc[2][M][NC];
#pragma unroll
    for (int i = 0; i < M; ++i) {
        ri[i] = row_info(a, b, PAGED ? old + a.Lq : len, r0 + ty + 16 * i);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            mx[m][i] = -INFINITY;
            sum[m][i] = 0.f;
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[m][i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    int j0 = split * a.keys_per_split, end = min(len, j0 + a.keys_per_split);
    if constexpr (PAGED) {
        // Shares of the sequence's own keys: the table is as wide as the longest's.
        const int per = ((len + a.splits - 1) / a.splits + KT - 1) / KT * KT;
        j0 = split * per;
        end = r0 < count * a.G ? min(len, j0 + per) : 0;
    }
    // Keys after the last row's query end the walk where positions are indices.
    if (a.causal && !a.pos_q && !a.pos_k) {
        const int last = static_cast<int>(a.div_G.div(min(r0 + QT, a.rows) - 1));
        end = min(end, (PAGED ? old : len - a.Lq) + last + 1);
    }
    const auto ask = [&](int of) {  // the rows of step `of`, whose infos are there
        const int *seen = infos + (of % 3 * 2 + 1) * KT;
        const int2 *where = at + of % 3 * KT;
#pragma unroll
        for (int m = 0; m < 2; ++m)
            ask_paged<T, DP>(a, a.k, n * a.ks[2] + m * a.ks[3], a.ks[0], a.ks[1], a.D, seen, where, ak[m]);
        ask_paged<T, F::WV>(a, a.v, n * a.vs[2], a.vs[0], a.vs[1], a.Dv, seen, where, av);
    };
    if constexpr (AHEAD) {
        for (int i = 0; i < 2; ++i) load_paged_info(a, b, end, j0 + i * KT, KT, infos + i * 2 * KT, infos + (i * 2 + 1) * KT, at + i * KT);
        __syncthreads();
        ask(0);
    }
    for (; j0 < end; j0 += KT, ++step) {
        __syncthreads();
        if constexpr (AHEAD) {
            kpos = infos + step % 3 * 2 * KT;
            kseen = kpos + KT;
#pragma unroll
            for (int m = 0; m < 2; ++m) put_paged<DP>(ak[m], sk + m * KT * (DP + 4));
            put_paged<F::WV>(av, sv);
            if (step > 0 && threadIdx.x < KT) {
                const int x = (step + 1) % 3;
                at[x * KT + threadIdx.x] = ahead.at;
                infos[(x * 2 + 1) * KT + threadIdx.x] = ahead.seen;
                infos[x * 2 * KT + threadIdx.x] = ahead.pos;
            }
        } else if constexpr (PAGED) {
            load_paged_info(a, b, end, j0, KT, kpos, kseen, at);
        } else {
            load_key_info(a, b, end, j0, KT, kpos, kseen);
        }
        __syncthreads();
        if constexpr (AHEAD) {
            ask(step + 1);
            if (threadIdx.x < KT) ahead = paged_key(a, b, end, j0 + 2 * KT + threadIdx.x);
        } else if constexpr (PAGED) {
            for (int m = 0; m < 2; ++m)
                load_paged<T, DP>(a, a.k, n * a.ks[2] + m * a.ks[3], a.ks[0], a.ks[1], KT, a.D, kseen, at, sk + m * KT * (DP + 4));
            load_paged<T, F::WV>(a, a.v, n * a.vs[2], a.vs[0], a.vs[1], KT, a.Dv, kseen, at, sv);
        } else {
            for (int m = 0; m < 2; ++m)
                load_keys<T, DP>(a, a.k, b * a.ks[0] + n * a.ks[2] + m * a.ks[3], a.ks[1], j0, KT, a.D, kseen, sk + m * KT * (DP + 4));
            load_keys<T, F::WV>(a, a.v, b * a.vs[0] + n * a.vs[2], a.vs[1], j0, KT, a.Dv, kseen, sv);
        }
        if constexpr (!AHEAD) __syncthreads();
        float bias[M][N];
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                int seen = kseen[tx + 16 * j];
                if constexpr (PAGED)
                    if (ri[i].l >= count || (a.pg.tree && seen && ri[i].l >= 0 && !tree_sees(a, b, ri[i].l, j0 + tx + 16 * j, old))) seen = 0;
                bias[i][j] = bias_of(a, bt, seen, kpos[tx + 16 * j] - ri[i].pos, ri[i].g);
            }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            float t[M][N];
            scores<M, N, DP>(sq + m * QT * (DP + 4), sk + m * KT * (DP + 4), ty, tx, t);
#pragma unroll
            for (int i = 0; i < M; ++i) {
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float s = fmaf(t[i][j], a.scale_log2, bias[i][j]);
                    t[i][j] = bias[i][j] == -INFINITY ? -INFINITY : s;
                    top = fmaxf(top, t[i][j]);
                }
                top = fmaxf(mx[m][i], row_max(top));
                const float base = top == -INFINITY ? 0.f : top;
                const float shrink = ex2(mx[m][i] - base);
                mx[m][i] = top;
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float p = ex2(t[i][j] - base);
                    s += p;
                    sp[(m * QT + ty + 16 * i) * (KT + 4) + tx + 16 * j] = p;
                }
                sum[m][i] = fmaf(sum[m][i], shrink, row_sum(s));
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    acc[m][i][c].x *= shrink;
                    acc[m][i][c].y *= shrink;
                    acc[m][i][c].z *= shrink;
                    acc[m][i][c].w *= shrink;
                }
            }
        }
        __syncwarp();  // a row's weights are written and read by one half-warp
#pragma unroll
        for (int m = 0; m < 2; ++m)
            products<M, KT, F::WV, NC>(sp + m * QT * (KT + 4), sv, ty, tx, acc[m]);
    }
#pragma unroll
    for (int i = 0; i < M; ++i) {
        if (ri[i].l < 0) continue;
        const int r = r0 + ty + 16 * i, h = n * a.G + ri[i].g;
        // A row that saw no key has no sums, not even 0 times a value that is not finite.
#pragma unroll
        for (int m = 0; m < 2; ++m)
            if (sum[m][i] == 0.f)
#pragma unroll
                for (int c = 0; c < NC; ++c) acc[m][i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (a.splits > 1) {
            const int64_t at = ((static_cast<int64_t>(b) * a.Hkv + n) * a.rows + r) * a.splits + split;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                if (tx == 0) {
                    a.part_ml[(at * 2 + m) * 2] = mx[m][i];
                    a.part_ml[(at * 2 + m) * 2 + 1] = sum[m][i];
                }
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const float x[4] = {acc[m][i][c].x, acc[m][i][c].y, acc[m][i][c].z, acc[m][i][c].w};
                    for (int e = 0; e < 4; ++e)
                        if (4 * tx + 64 * c + e < a.Dv) a.part_o[(at * 2 + m) * a.Dv + 4 * tx + 64 * c + e] = x[e];
                }
            }
            continue;
        }
        const float w0 = sum[0][i] == 0.f ? 0.f : 1.f / sum[0][i];
        const float w1 = sum[1][i] == 0.f ? 0.f : 1.f / sum[1][i];
        const float lam = sum[1][i] == 0.f ? 0.f : a.lam[h];
        const int64_t row = (static_cast<int64_t>(b) * a.Lq + ri[i].l) * a.H + h;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const float x[4] = {acc[0][i][c].x, acc[0][i][c].y, acc[0][i][c].z, acc[0][i][c].w};
            const float y[4] = {acc[1][i][c].x, acc[1][i][c].y, acc[1][i][c].z, acc[1][i][c].w};
            for (int e = 0; e < 4; ++e) {
                const int d = 4 * tx + 64 * c + e;
                if (d < a.Dv) dattn_store<T>(a, row, d, x[e] * w0 - lam * (y[e] * w1), y[e] * w1);
            }
        }
        if (a.lse && tx < 2)
            a.lse[((static_cast<int64_t>(b) * a.H + h) * 2 + tx) * a.Lq + ri[i].l] =
                tx ? (sum[1][i] == 0.f ? INFINITY : mx[1][i] + log2f(sum[1][i]))
                   : (sum[0][i] == 0.f ? INFINITY : mx[0][i] + log2f(sum[0][i]));
    }
}

int padded_width(const DattnArgs &a)
{
    const int w = a.Dv > 2 * a.D ? (a.Dv + 1) / 2 : a.D;
    return w <= 32 ? 32 : w <= 64 ? 64 : 128;
}

size_t table_floats(const DattnArgs &a) { return a.nb ? a.nb * a.G + (2 * a.reach + 2) / 2 + 2 : 0; }

constexpr size_t kTableFloats = DATTN_MAX_TABLE + (2 * DATTN_MAX_REACH + 2) / 2 + 2;  // at most

template <typename K> cudaError_t launch(K kernel, dim3 grid, size_t floats, size_t most, const DattnArgs &a, cudaStream_t st)
{
    const cudaError_t e = allow_shared(kernel, most * sizeof(float));
    if (e != cudaSuccess) return e;
    kernel<<<grid, kThreadsG, floats * sizeof(float), st>>>(a);
    return cudaGetLastError();
}

template <typename T, int DP, bool PAGED> cudaError_t forward_width(const DattnArgs &a, cudaStream_t st)
{
    const int qt = dattn_general_row_tile(a);
    const dim3 grid(static_cast<unsigned>((a.rows + qt - 1) / qt * a.splits), a.Hkv, a.B);
    constexpr size_t few = FwdTile<T, DP, 16>::floats, many = FwdTile<T, DP, 64>::floats;
    if (qt == 16) return launch(dattn_fwd_kernel<T, DP, 16, PAGED>, grid, few + table_floats(a), few + kTableFloats, a, st);
    return launch(dattn_fwd_kernel<T, DP, 64, PAGED>, grid, many + table_floats(a), many + kTableFloats, a, st);
}

}  // namespace
}  // namespace da
