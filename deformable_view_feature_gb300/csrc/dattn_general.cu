// Differential attention (include/dattn.h) on the fp32 units: every type,
// width, stride and alignment. fp32 inputs always come here (the tensor cores
// round their operands to at most 11 bits); 16-bit inputs only where the
// tensor-core kernels' rule on widths and alignment sends them.
//
// One CTA of 256 threads takes a tile of rows (queries x the heads that share
// a key head) and walks over the keys, both maps at once, with the running
// maximum and sum of each softmax in registers, so no score is ever stored.
// Threads form a 16 x 16 grid; thread (ty, tx) owns rows ty + 16 i and, of a
// score tile, columns tx + 16 j, or of an output tile the four channels at
// 4 tx + 64 c. All shared tiles are row-major with a pad of four floats:
// sixteen neighbouring rows then fall on different banks in 16-byte reads, and
// both products read their operands along a row, 64 multiply-adds to eight
// 16-byte reads. 900 x 900 rows of 4 heads, D = 32, fp32: 55 us for 0.83
// GFLOP counted once, some 15 TFLOP/s; two CTAs per SM hide part of each
// other's loads and of the latency between the two products.
#include "dattn_general.cuh"

namespace da {
namespace {

// Joins the parts of a row that was split over the keys: one warp per row.
template <typename T> __global__ void __launch_bounds__(kThreadsG) dattn_merge_kernel(const __grid_constant__ DattnArgs a)
{
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreadsG / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int64_t bn = row / a.rows;
    if (bn >= static_cast<int64_t>(a.B) * a.Hkv) return;
    const int r = static_cast<int>(row - bn * a.rows), b = static_cast<int>(bn / a.Hkv), n = static_cast<int>(bn - b * a.Hkv);
    const int l = static_cast<int>(a.div_G.div(r)), h = n * a.G + r - l * a.G;
    const float *ml = a.part_ml + row * a.splits * 4, *po = a.part_o + row * a.splits * 2 * a.Dv;
    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f}, inv[2];
    for (int s = 0; s < a.splits; ++s)
        for (int m = 0; m < 2; ++m) top[m] = fmaxf(top[m], ml[(s * 2 + m) * 2]);
    for (int m = 0; m < 2; ++m) {
        const float base = top[m] == -INFINITY ? 0.f : top[m];
        for (int s = 0; s < a.splits; ++s) sum[m] = fmaf(ml[(s * 2 + m) * 2 + 1], ex2(ml[(s * 2 + m) * 2] - base), sum[m]);
        inv[m] = sum[m] == 0.f ? 0.f : 1.f / sum[m];
        if (a.lse && lane == m)
            a.lse[((static_cast<int64_t>(b) * a.H + h) * 2 + m) * a.Lq + l] = sum[m] == 0.f ? INFINITY : top[m] + log2f(sum[m]);
        top[m] = base;
    }
    const float lam = sum[1] == 0.f ? 0.f : a.lam[h];  // parts of a row without keys are zeros
    const int64_t orow = (static_cast<int64_t>(b) * a.Lq + l) * a.H + h;
    for (int d = lane; d < a.Dv; d += 32) {
        float o[2] = {0.f, 0.f};
        for (int s = 0; s < a.splits; ++s)
            for (int m = 0; m < 2; ++m)
                o[m] = fmaf(po[(s * 2 + m) * a.Dv + d], ex2(ml[(s * 2 + m) * 2] - top[m]), o[m]);
        dattn_store<T>(a, orow, d, o[0] * inv[0] - lam * (o[1] * inv[1]), o[1] * inv[1]);
    }
}

// ---- backward --------------------------------------------------------------

template <typename T, int DP> struct BwdTile {
    static constexpr int RT = DP <= 64 ? 64 : 32, KT = RT;
    static constexpr int WV = 2 * DP;
    static constexpr int M = RT / 16, N = KT / 16, NV = WV / 64, ND = DP < 64 ? 1 : DP / 64;
    static constexpr int q = 0, g = q + 2 * RT * (DP + 4), k = g + RT * (WV + 4), v = k + 2 * KT * (DP + 4),
                         s = v + KT * (WV + 4), info = s + 3 * RT * (KT + 4), floats = info + 2 * KT + 7 * RT;
};

// grad_q, and the exact d_m of dattn.h. The d_m that s_m needs comes from the
// saved outputs, which hold 16 bits or more; the walk over the keys then gives
// the remainder, sum_j s_m, in fp32.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreadsG) dattn_grad_q_kernel(const __grid_constant__ DattnArgs a)
{
    using F = BwdTile<T, DP>;
    constexpr int M = F::M, N = F::N, KT = F::KT, QT = F::RT;
    extern __shared__ float sm[];
    float *sq = sm + F::q, *sg = sm + F::g, *sk = sm + F::k, *sv = sm + F::v, *ss = sm + F::s;
    int *kpos = reinterpret_cast<int *>(sm + F::info), *kseen = kpos + KT;
    const BiasTable bt{sm + F::floats, reinterpret_cast<uint16_t *>(sm + F::floats + a.nb * a.G)};
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int tile = blockIdx.x / a.splits, split = blockIdx.x - tile * a.splits;
    const int n = blockIdx.y, b = blockIdx.z, r0 = tile * QT;
    const int len = dattn_length(a, b);
    const int64_t ob = static_cast<int64_t>(b) * a.Lq * a.H * a.Dv;  // of out-like tensors

    load_bias(a, n, bt);
    for (int m = 0; m < 2; ++m)
        load_rows<T, DP>(a, a.q, b * a.qs[0] + m * a.qs[3], a.qs[1], a.qs[2], n, r0, QT, a.D, sq + m * QT * (DP + 4));
    load_rows<T, F::WV>(a, a.grad_out, ob, static_cast<int64_t>(a.H) * a.Dv, a.Dv, n, r0, QT, a.Dv, sg);
    __syncthreads();
    RowInfo ri[M];
    float lse[2][M], dl[2][M], rest[2][M], lam[M];
    float4 acc[2][M][F::ND];
#pragma unroll
    for (int i = 0; i < M; ++i) {
        ri[i] = row_info(a, b, len, r0 + ty + 16 * i);
        const int h = n * a.G + ri[i].g;
        lam[i] = a.lam[h];
        float d0 = 0.f, d1 = 0.f;
        if (ri[i].l >= 0) {
            const int64_t row = (static_cast<int64_t>(b) * a.Lq + ri[i].l) * a.H + h;
            const T *out = static_cast<const T *>(a.out) + row * a.Dv, *save = static_cast<const T *>(a.out1) + row * kSaved<T> * a.Dv;
            for (int d = tx; d < a.Dv; d += 16) {
                const float gv = sg[(ty + 16 * i) * (F::WV + 4) + d];
                if constexpr (sizeof(T) == 2) {
                    d0 = fmaf(gv, dattn_whole(out[d], save[d]), d0);
                    d1 = fmaf(gv, dattn_whole(save[a.Dv + d], save[2 * a.Dv + d]), d1);
                } else {
                    d0 = fmaf(gv, out[d], d0);
                    d1 = fmaf(gv, save[d], d1);
                }
            }
        }
        dl[1][i] = row_sum(d1);
        dl[0][i] = fmaf(lam[i], dl[1][i], row_sum(d0));  // out = o_0 - lam o_1
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            lse[m][i] = ri[i].l < 0 ? INFINITY : a.lse[((static_cast<int64_t>(b) * a.H + h) * 2 + m) * a.Lq + ri[i].l];
            rest[m][i] = 0.f;
            if (lse[m][i] == INFINITY) dl[m][i] = 0.f;  // sees no key: whatever grad_out holds there is not used
#pragma unroll
            for (int c = 0; c < F::ND; ++c) acc[m][i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    int end = len;
    const bool steps_down = a.causal && !a.pos_q && !a.pos_k;  // a query sees the keys up to its own index
    if (steps_down) end = min(end, len - a.Lq + static_cast<int>(a.div_G.div(min(r0 + QT, a.rows) - 1)) + 1);
    int begin = 0;
    if (a.mask) {  // from the first tile with a key to be used to the last such key
        __shared__ int first_used, last_used;
        const uint8_t *mask = a.mask + static_cast<int64_t>(b) * a.Lk;
        if (threadIdx.x == 0) {
            first_used = INT32_MAX;
            last_used = -1;
        }
        __syncthreads();
        for (int i = 0; i < end; i += kThreadsG) {
            const int j = i + static_cast<int>(threadIdx.x);
            const bool use = j < end && mask[j];
            if (use) atomicMin(&first_used, j);
            if (__syncthreads_or(use)) break;
        }
        for (int i = end - 1; i >= 0; i -= kThreadsG) {
            const int j = i - static_cast<int>(threadIdx.x);
            const bool use = j >= 0 && mask[j];
            if (use) atomicMax(&last_used, j);
            if (__syncthreads_or(use)) break;
        }
        begin = last_used < 0 ? 0 : first_used / KT * KT;
        end = last_used + 1;
    }
    // Whether the first tile holds all keys that a row of the tile sees; the
    // split that has it then knows the rows' d_m best.
    const bool one = end <= begin + KT, some = one || (steps_down && len - a.Lq + static_cast<int>(a.div_G.div(r0)) < begin + KT);
    const int writer = begin / a.keys_per_split, first = max(begin, split * a.keys_per_split);
    end = min(end, (split + 1) * a.keys_per_split);
    for (int j0 = first; j0 < end; j0 += KT) {
        __syncthreads();
        load_key_info(a, b, end, j0, KT, kpos, kseen);
        __syncthreads();
        for (int m = 0; m < 2; ++m)
            load_keys<T, DP>(a, a.k, b * a.ks[0] + n * a.ks[2] + m * a.ks[3], a.ks[1], j0, KT, a.D, kseen, sk + m * KT * (DP + 4));
        load_keys<T, F::WV>(a, a.v, b * a.vs[0] + n * a.vs[2], a.vs[1], j0, KT, a.Dv, kseen, sv);
        __syncthreads();
        float e[M][N];
        scores<M, N, F::WV>(sg, sv, ty, tx, e);
        float bias[M][N];
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) bias[i][j] = bias_of(a, bt, kseen[tx + 16 * j], kpos[tx + 16 * j] - ri[i].pos, ri[i].g);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            float t[M][N];
            scores<M, N, DP>(sq + m * QT * (DP + 4), sk + m * KT * (DP + 4), ty, tx, t);
#pragma unroll
            for (int i = 0; i < M; ++i) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const bool on = bias[i][j] != -INFINITY && lse[m][i] != INFINITY;
                    t[i][j] = on ? ex2(fmaf(t[i][j], a.scale_log2, bias[i][j] - lse[m][i])) : 0.f;
                }
                if (j0 == begin && some) {
                    // All of a whole row's keys are here: weights that sum to 1
                    // and d_m from them, so that a row of one key gives exactly
                    // 0. (The whole warp takes this way: its rows' sums are
                    // formed by shuffles.)
                    const bool whole = one || ri[i].pos < begin + KT;
                    float z = 0.f, d = 0.f;
#pragma unroll
                    for (int j = 0; j < N; ++j) z += t[i][j];
                    z = row_sum(z);
                    if (!whole) z = 1.f;
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        t[i][j] = z == 0.f ? 0.f : t[i][j] / z;
                        d += t[i][j] != 0.f ? t[i][j] * e[i][j] : 0.f;
                    }
                    d = row_sum(d);
                    if (whole) dl[m][i] = d;
                }
                float r = 0.f;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float s = t[i][j] != 0.f ? t[i][j] * (e[i][j] - dl[m][i]) : 0.f;
                    r += s;
                    ss[(m * QT + ty + 16 * i) * (KT + 4) + tx + 16 * j] = m ? -lam[i] * s : s;
                }
                rest[m][i] += row_sum(r);
            }
        }
        __syncwarp();
#pragma unroll
        for (int m = 0; m < 2; ++m)
            products<M, KT, DP, F::ND>(ss + m * QT * (KT + 4), sk + m * KT * (DP + 4), ty, tx, acc[m]);
    }
#pragma unroll
    for (int i = 0; i < M; ++i) {
        if (ri[i].l < 0) continue;
        const int r = r0 + ty + 16 * i, h = n * a.G + ri[i].g;
        const int64_t row = (static_cast<int64_t>(b) * a.Hkv + n) * a.rows + r;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            // A row that sees no key has no gradient, not even 0 times a key or lam that is not finite.
            if (lse[m][i] == INFINITY)
#pragma unroll
                for (int c = 0; c < F::ND; ++c) acc[m][i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
            float *delta = a.delta + ((static_cast<int64_t>(b) * a.Hkv + n) * 2 + m) * a.rows + r;
            if (tx == 0) {
                if (a.splits == 1) *delta = dl[m][i] + rest[m][i];
                else if (split == writer) *delta = dl[m][i];
                if (a.splits > 1) a.part_ml[(row * a.splits + split) * 2 + m] = rest[m][i];
            }
            const int64_t at = (((static_cast<int64_t>(b) * a.Lq + ri[i].l) * a.H + h) * 2 + m) * a.D;
#pragma unroll
            for (int c = 0; c < F::ND; ++c) {
                const float x[4] = {acc[m][i][c].x, acc[m][i][c].y, acc[m][i][c].z, acc[m][i][c].w};
                for (int e = 0; e < 4; ++e) {
                    const int d = 4 * tx + 64 * c + e;
                    if (d >= a.D) continue;
                    if (a.splits > 1) a.part_o[((row * a.splits + split) * 2 + m) * a.D + d] = x[e];
                    else static_cast<T *>(a.grad_q)[at + d] = dattn_round<T>(x[e] * a.scale);
                }
            }
        }
    }
}

// Joins the parts of grad_q and of the d_m: one warp per row.
template <typename T> __global__ void __launch_bounds__(kThreadsG) dattn_join_q_kernel(const __grid_constant__ DattnArgs a)
{
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreadsG / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int64_t bn = row / a.rows;
    if (bn >= static_cast<int64_t>(a.B) * a.Hkv) return;
    const int r = static_cast<int>(row - bn * a.rows), b = static_cast<int>(bn / a.Hkv), n = static_cast<int>(bn - b * a.Hkv);
    const int l = static_cast<int>(a.div_G.div(r)), h = n * a.G + r - l * a.G;
    if (lane < 2) {
        float s = 0.f;
        for (int k = 0; k < a.splits; ++k) s += a.part_ml[(row * a.splits + k) * 2 + lane];
        a.delta[(bn * 2 + lane) * a.rows + r] += s;
    }
    T *dst = static_cast<T *>(a.grad_q) + ((static_cast<int64_t>(b) * a.Lq + l) * a.H + h) * 2 * a.D;
    for (int d = lane; d < 2 * a.D; d += 32) {
        float s = 0.f;
        for (int k = 0; k < a.splits; ++k) s += a.part_o[(row * a.splits + k) * 2 * a.D + d];
        dst[d] = dattn_round<T>(s * a.scale);
    }
}

// grad_k, grad_v and the tile's share of grad_table. Roles are exchanged: a
// CTA owns a tile of keys and walks over the rows, of all heads that share the
// key head.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreadsG) dattn_grad_kv_kernel(const __grid_constant__ DattnArgs a)
{
    using F = BwdTile<T, DP>;
    constexpr int M = F::M, N = F::N, KT = F::KT, RT = F::RT;
    extern __shared__ float sm[];
    float *sq = sm + F::q, *sg = sm + F::g, *sk = sm + F::k, *sv = sm + F::v, *ss = sm + F::s;
    int *kpos = reinterpret_cast<int *>(sm + F::info), *kseen = kpos + KT;
    int *rpos = kseen + KT, *rg = rpos + RT;
    float *rlse = reinterpret_cast<float *>(rg + RT), *rdl = rlse + 2 * RT, *rlam = rdl + 2 * RT;
    const BiasTable bt{sm + F::floats, reinterpret_cast<uint16_t *>(sm + F::floats + a.nb * a.G)};
    // Each thread's sums per bucket and head, or each warp's where shared memory
    // does not hold 256 of them. (Warps' sums take a walk over the distinct
    // buckets of every 32 scores: 160 us against 111 for the backward pass at
    // 333 tokens, 32 buckets, 3 heads to a key head.)
    const bool own_sums = a.own_sums;
    float *all_sums = sm + F::floats + bias_floats(a.nb, a.G, a.reach);
    float *sums = all_sums + (own_sums ? threadIdx.x : (threadIdx.x >> 5) * a.nb * a.G);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, lane = threadIdx.x & 31;
    const int tile = blockIdx.x / a.row_splits, split = blockIdx.x - tile * a.row_splits;
    const int n = blockIdx.y, b = blockIdx.z, j0 = tile * KT;
    const int len = dattn_length(a, b);
    const int64_t ob = static_cast<int64_t>(b) * a.Lq * a.H * a.Dv;

    load_bias(a, n, bt);
    if (own_sums)
        for (int i = 0; i < a.nb * a.G; ++i) sums[i * kThreadsG] = 0.f;
    else
        for (int i = lane; i < a.nb * a.G; i += 32) sums[i] = 0.f;
    load_key_info(a, b, len, j0, KT, kpos, kseen);
    __syncthreads();
    for (int m = 0; m < 2; ++m)
        load_keys<T, DP>(a, a.k, b * a.ks[0] + n * a.ks[2] + m * a.ks[3], a.ks[1], j0, KT, a.D, kseen, sk + m * KT * (DP + 4));
    load_keys<T, F::WV>(a, a.v, b * a.vs[0] + n * a.vs[2], a.vs[1], j0, KT, a.Dv, kseen, sv);
    float4 gv[M][F::NV], gk[2][M][F::ND];
#pragma unroll
    for (int i = 0; i < M; ++i) {
#pragma unroll
        for (int c = 0; c < F::NV; ++c) gv[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < F::ND; ++c) gk[0][i][c] = gk[1][i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    int first = 0;
    // The first query that sees the tile's first key, where positions are indices.
    if (a.causal && !a.pos_q && !a.pos_k) first = min(max(j0 - (len - a.Lq), 0), a.Lq) * a.G;
    // This CTA's share of the rows, in whole tiles.
    const int steps = (a.rows - first + RT - 1) / RT, share = (steps + a.row_splits - 1) / a.row_splits * RT;
    first += split * share;
    const int last = j0 < len ? min(a.rows, first + share) : 0;
    for (int r0 = first; r0 < last; r0 += RT) {
        __syncthreads();
        for (int i = threadIdx.x; i < RT; i += kThreadsG) {
            const RowInfo ri = row_info(a, b, len, r0 + i);
            const int h = n * a.G + ri.g;
            rpos[i] = ri.pos;
            rg[i] = ri.g;
            rlam[i] = a.lam[h];
            for (int m = 0; m < 2; ++m) {
                rlse[2 * i + m] = ri.l < 0 ? INFINITY : a.lse[((static_cast<int64_t>(b) * a.H + h) * 2 + m) * a.Lq + ri.l];
                rdl[2 * i + m] = ri.l < 0 ? 0.f : a.delta[((static_cast<int64_t>(b) * a.Hkv + n) * 2 + m) * a.rows + r0 + i];
            }
        }
        for (int m = 0; m < 2; ++m)
            load_rows<T, DP>(a, a.q, b * a.qs[0] + m * a.qs[3], a.qs[1], a.qs[2], n, r0, RT, a.D, sq + m * RT * (DP + 4));
        load_rows<T, F::WV>(a, a.grad_out, ob, static_cast<int64_t>(a.H) * a.Dv, a.Dv, n, r0, RT, a.Dv, sg);
        __syncthreads();
        // A row that sees no key takes no part, whatever q and grad_out hold there.
        for (int i = threadIdx.x; i < RT * F::WV; i += kThreadsG) {
            const int row = i / F::WV, d = i - row * F::WV;
            if (rlse[2 * row] == INFINITY) {
                sg[row * (F::WV + 4) + d] = 0.f;
                sq[(d / DP) * RT * (DP + 4) + row * (DP + 4) + d % DP] = 0.f;
            }
        }
        __syncthreads();
        float e[M][N], both[M][N], bias[M][N];
        scores<M, N, F::WV>(sv, sg, ty, tx, e);
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j)
                bias[i][j] = bias_of(a, bt, kseen[ty + 16 * i], kpos[ty + 16 * i] - rpos[tx + 16 * j], rg[tx + 16 * j]);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            float t[M][N];
            scores<M, N, DP>(sk + m * KT * (DP + 4), sq + m * RT * (DP + 4), ty, tx, t);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int c = tx + 16 * j;
                const float lse = rlse[2 * c + m], dl = rdl[2 * c + m], f = m ? -rlam[c] : 1.f;
#pragma unroll
                for (int i = 0; i < M; ++i) {
                    const bool on = bias[i][j] != -INFINITY && lse != INFINITY;
                    const float p = on ? f * ex2(fmaf(t[i][j], a.scale_log2, bias[i][j] - lse)) : 0.f, s = on ? p * (e[i][j] - dl) : 0.f;
                    float *w = ss + (ty + 16 * i) * (RT + 4) + c;
                    w[0] = m ? w[0] + p : p;
                    w[(1 + m) * KT * (RT + 4)] = s;
                    both[i][j] = m ? both[i][j] + s : s;
                }
            }
        }
        __syncwarp();
        products<M, RT, F::WV, F::NV>(ss, sg, ty, tx, gv);
#pragma unroll
        for (int m = 0; m < 2; ++m)
            products<M, RT, DP, F::ND>(ss + (1 + m) * KT * (RT + 4), sq + m * RT * (DP + 4), ty, tx, gk[m]);
        if (a.nb && own_sums) {
#pragma unroll
            for (int i = 0; i < M; ++i)
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int c = tx + 16 * j;
                    sums[(bucket_of(a, bt, kpos[ty + 16 * i] - rpos[c]) * a.G + rg[c]) * kThreadsG] += both[i][j];
                }
        } else if (a.nb) {
            // The warp's sums per bucket, bucket by bucket in the order of
            // its lanes: no atomics, so the order is the same in every run.
#pragma unroll
            for (int i = 0; i < M; ++i)
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int c = tx + 16 * j;
                    const int at = bucket_of(a, bt, kpos[ty + 16 * i] - rpos[c]) * a.G + rg[c];
                    unsigned left = 0xffffffffu;
                    while (left) {
                        const int who = __shfl_sync(0xffffffffu, at, __ffs(left) - 1);
                        const unsigned same = __ballot_sync(0xffffffffu, at == who);
                        float s = at == who ? both[i][j] : 0.f;
#pragma unroll
                        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                        if (lane == 0) sums[who] += s;
                        left &= ~same;
                    }
                }
        }
    }
#pragma unroll
    for (int i = 0; i < M; ++i) {
        const int j = j0 + ty + 16 * i;
        if (j >= a.Lk) continue;
        const int64_t at = (static_cast<int64_t>(b) * a.Lk + j) * a.Hkv + n;
        float *part = a.row_splits > 1 ? a.part_kv + (at * a.row_splits + split) * (a.Dv + 2 * a.D) : nullptr;
#pragma unroll
        for (int c = 0; c < F::NV; ++c) {
            const float x[4] = {gv[i][c].x, gv[i][c].y, gv[i][c].z, gv[i][c].w};
            for (int e = 0; e < 4; ++e)
                if (4 * tx + 64 * c + e < a.Dv) {
                    if (part) part[4 * tx + 64 * c + e] = x[e];
                    else static_cast<T *>(a.grad_v)[at * a.Dv + 4 * tx + 64 * c + e] = dattn_round<T>(x[e]);
                }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int c = 0; c < F::ND; ++c) {
                const float x[4] = {gk[m][i][c].x, gk[m][i][c].y, gk[m][i][c].z, gk[m][i][c].w};
                for (int e = 0; e < 4; ++e)
                    if (4 * tx + 64 * c + e < a.D) {
                        if (part) part[a.Dv + m * a.D + 4 * tx + 64 * c + e] = x[e];
                        else static_cast<T *>(a.grad_k)[(at * 2 + m) * a.D + 4 * tx + 64 * c + e] = dattn_round<T>(x[e] * a.scale);
                    }
            }
    }
    if (a.nb) {
        __syncthreads();
        float *out = a.part_table + ((static_cast<int64_t>(b) * a.Hkv + n) * a.table_ctas + blockIdx.x) * a.nb * a.G;
        if (own_sums) {
            for (int i = threadIdx.x >> 5; i < a.nb * a.G; i += kThreadsG / 32) {
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < kThreadsG / 32; ++w) s += all_sums[i * kThreadsG + w * 32 + lane];
#pragma unroll
                for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                if (lane == 0) out[i] = s;
            }
        } else {
            for (int i = threadIdx.x; i < a.nb * a.G; i += kThreadsG) {
                float s = 0.f;
                for (int w = 0; w < kThreadsG / 32; ++w) s += all_sums[w * a.nb * a.G + i];
                out[i] = s;
            }
        }
    }
}

// Joins the parts of grad_v and grad_k: one warp per key and key head.
template <typename T> __global__ void __launch_bounds__(kThreadsG) dattn_join_kv_kernel(const __grid_constant__ DattnArgs a)
{
    const int64_t at = static_cast<int64_t>(blockIdx.x) * (kThreadsG / 32) + (threadIdx.x >> 5);
    if (at >= static_cast<int64_t>(a.B) * a.Lk * a.Hkv) return;
    const int width = a.Dv + 2 * a.D;
    for (int d = threadIdx.x & 31; d < width; d += 32) {
        float s = 0.f;
        for (int k = 0; k < a.row_splits; ++k) s += a.part_kv[(at * a.row_splits + k) * width + d];
        if (d < a.Dv) static_cast<T *>(a.grad_v)[at * a.Dv + d] = dattn_round<T>(s);
        else static_cast<T *>(a.grad_k)[at * 2 * a.D + d - a.Dv] = dattn_round<T>(s * a.scale);
    }
}

// grad_lam[h] and grad_table[n, h]: one CTA per (key head, sum), the terms in
// a fixed order.
__global__ void __launch_bounds__(kThreadsG) dattn_finish_kernel(const __grid_constant__ DattnArgs a)
{
    __shared__ double sh[kThreadsG];
    const int n = blockIdx.y, i = blockIdx.x;
    double s = 0.0;
    float *dst;
    if (i < a.G) {
        dst = a.grad_lam + n * a.G + i;
        for (int b = 0; b < a.B; ++b) {
            const float *d = a.delta + ((static_cast<int64_t>(b) * a.Hkv + n) * 2 + 1) * a.rows + i;
            for (int l = threadIdx.x; l < a.Lq; l += kThreadsG) s -= d[static_cast<int64_t>(l) * a.G];
        }
    } else {
        const int e = i - a.G, bucket = e / a.G, g = e - bucket * a.G;
        dst = a.grad_table + static_cast<int64_t>(bucket) * a.H + n * a.G + g;
        for (int c = threadIdx.x; c < a.B * a.table_ctas; c += kThreadsG) {
            const int b = c / a.table_ctas;
            s += a.part_table[((static_cast<int64_t>(b) * a.Hkv + n) * a.table_ctas + (c - b * a.table_ctas)) * a.nb * a.G + e];
        }
    }
    sh[threadIdx.x] = s;
    __syncthreads();
    for (int o = kThreadsG / 2; o; o >>= 1) {
        if (static_cast<int>(threadIdx.x) < o) sh[threadIdx.x] += sh[threadIdx.x + o];
        __syncthreads();
    }
    if (threadIdx.x == 0) *dst = static_cast<float>(sh[0]);
}

template <typename T, int DP> cudaError_t backward_width(const DattnArgs &a, cudaStream_t st)
{
    using F = BwdTile<T, DP>;
    cudaError_t e = cudaSuccess;
    const int warps = kThreadsG / 32;
    if (a.rows > 0) {
        const dim3 grid(static_cast<unsigned>((a.rows + F::RT - 1) / F::RT * a.splits), a.Hkv, a.B);
        e = launch(dattn_grad_q_kernel<T, DP>, grid, F::floats + table_floats(a), F::floats + kTableFloats, a, st);
        if (e == cudaSuccess && a.splits > 1) {
            const int64_t rows = static_cast<int64_t>(a.B) * a.Hkv * a.rows;
            dattn_join_q_kernel<T><<<static_cast<unsigned>((rows + warps - 1) / warps), kThreadsG, 0, st>>>(a);
            e = cudaGetLastError();
        }
    }
    if (e == cudaSuccess && a.Lk > 0) {
        const dim3 grid(static_cast<unsigned>((a.Lk + F::KT - 1) / F::KT * a.row_splits), a.Hkv, a.B);
        const size_t base = F::floats + table_floats(a), own = base + kThreadsG * a.nb * a.G;
        DattnArgs with = a;
        constexpr size_t most = 227 * 1024 / sizeof(float);
        with.own_sums = own <= most;
        e = launch(dattn_grad_kv_kernel<T, DP>, grid, with.own_sums ? own : base + warps * a.nb * a.G, most, with, st);
        if (e == cudaSuccess && a.row_splits > 1) {
            const int64_t keys = static_cast<int64_t>(a.B) * a.Lk * a.Hkv;
            dattn_join_kv_kernel<T><<<static_cast<unsigned>((keys + warps - 1) / warps), kThreadsG, 0, st>>>(a);
            e = cudaGetLastError();
        }
    }
    return e;
}

template <typename T> cudaError_t any_width(const DattnArgs &a, bool backward, cudaStream_t st)
{
    switch (padded_width(a)) {
    case 32: return backward ? backward_width<T, 32>(a, st) : forward_width<T, 32, false>(a, st);
    case 64: return backward ? backward_width<T, 64>(a, st) : forward_width<T, 64, false>(a, st);
    default: return backward ? backward_width<T, 128>(a, st) : forward_width<T, 128, false>(a, st);
    }
}

cudaError_t any_type(const DattnArgs &a, int dtype, bool backward, cudaStream_t st)
{
    switch (dtype) {
    case DA_F32: return any_width<float>(a, backward, st);
    case DA_BF16: return any_width<__nv_bfloat16>(a, backward, st);
    default: return any_width<__half>(a, backward, st);
    }
}

}  // namespace

// Sixteen rows or fewer per key head (single tokens) take a 16-row tile.
int dattn_general_row_tile(const DattnArgs &a) { return a.rows <= 16 ? 16 : 64; }
int dattn_general_tile(const DattnArgs &a) { return padded_width(a) <= 64 ? 64 : 32; }

cudaError_t dattn_forward_general(const DattnArgs &a, int dtype, cudaStream_t st) { return any_type(a, dtype, false, st); }

cudaError_t dattn_backward_general(const DattnArgs &a, int dtype, cudaStream_t st) { return any_type(a, dtype, true, st); }

cudaError_t dattn_merge(const DattnArgs &a, int dtype, cudaStream_t st)
{
    const int64_t rows = static_cast<int64_t>(a.B) * a.Hkv * a.rows;
    const unsigned grid = static_cast<unsigned>((rows + kThreadsG / 32 - 1) / (kThreadsG / 32));
    if (dtype == DA_F32) dattn_merge_kernel<float><<<grid, kThreadsG, 0, st>>>(a);
    else if (dtype == DA_BF16) dattn_merge_kernel<__nv_bfloat16><<<grid, kThreadsG, 0, st>>>(a);
    else dattn_merge_kernel<__half><<<grid, kThreadsG, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t dattn_finish_backward(const DattnArgs &a, cudaStream_t st)
{
    dattn_finish_kernel<<<dim3(a.G + a.nb * a.G, a.Hkv), kThreadsG, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace da
