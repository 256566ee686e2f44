// Differential attention over a paged cache on the fp32 units for few rows
// (include/paged.h): single tokens, of every type, width, stride and alignment.
// fp32 caches always come here or to the tiles of paged_general.cu.
//
// A key is used for little arithmetic, so nothing is staged: a warp reads its keys'
// rows straight into registers, half its lanes map 0's key and half map 1's, all of them the
// value, and holds the running maxima, sums and outputs of R rows. The dot
// products of KB keys with R rows, KB * R <= 16, are 16 sums over the 16 lanes of
// a half-warp; folded together they take 15 exchanges and leave each lane one
// (key, row) score of its map, which is where biases, masks and the exponential
// are applied, once. Sixteen warps to an SM (eight with 8 rows, whose registers
// leave room for one CTA) have KB keys each under way.
//
// Four ragged caches of up to 8,192 keys (2 key heads, D = 64, Dv = 128, a token
// of 8 heads; 55 MB) take 26 us in fp32, the tiles of paged_general.cu 73; with 8
// rows 55 us. That is 2.1 and 1.0 TB/s of the 6.8 of a copy: not memory bounds it
// but a batch's exchanges, for 4 keys and 4 rows 8 of pages and places, 15 to fold
// and 32 to spread the weights, which grow with the rows.
#include <cfloat>

#include "paged_internal.cuh"

namespace da {
namespace {

constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32;

// V elements as floats; zeros past the width.
template <typename T, int V> __device__ __forceinline__ void load_row(const T *row, int d, int width, float (&x)[V])
{
    if constexpr (V == 4 && sizeof(T) == 4) {
        const float4 v = d < width ? __ldcs(reinterpret_cast<const float4 *>(row + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
        x[0] = v.x;
        x[1] = v.y;
        x[2] = v.z;
        x[3] = v.w;
    } else if constexpr (V == 4) {
        const uint2 v = d < width ? __ldcs(reinterpret_cast<const uint2 *>(row + d)) : make_uint2(0, 0);
        const T *e = reinterpret_cast<const T *>(&v);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = dattn_float(e[i]);
    } else {
        x[0] = d < width ? dattn_float(row[d]) : 0.f;
    }
}

// Sums of 16 values over the 16 lanes of each half-warp: lane i of a half is
// left with the sum of value i.
__device__ __forceinline__ float fold16(float (&v)[16], int lane)
{
#pragma unroll
    for (int o = 8, n = 8; o; o >>= 1, n >>= 1)
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const bool up = lane & o;
            const float keep = up ? v[i + n] : v[i], send = up ? v[i] : v[i + n];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    return v[0];
}

// R rows, KB keys at once; V elements to a load; NK and NV loads to a row of a
// key and of a value.
template <typename T, int R, int KB, int V, int NK, int NV>
__global__ void __launch_bounds__(kFewThreads, R == 8 ? 1 : 2) paged_few_kernel(const __grid_constant__ DattnArgs a)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, m = lane >> 4, sub = lane & 15;
    const int groups = (a.rows + R - 1) / R;
    const int split = blockIdx.x % a.splits, r0 = blockIdx.x / a.splits % groups * R, n = blockIdx.y, b = blockIdx.z;
    const int len = dattn_length(a, b), count = paged_count(a, b), old = len - count;
    // Shares of the sequence's own keys, in whole turns of a warp.
    const int per = ((len + a.splits - 1) / a.splits + 31) / 32 * 32;
    int jb = split * per, end = min(len, jb + per);
    if (r0 >= count * a.G) end = 0;
    if (a.causal && !a.pos_q && !a.pos_k) {
        const int last = static_cast<int>(a.div_G.div(min(r0 + R, a.rows) - 1));
        end = min(end, old + last + 1);
    }

    float q[R][NK][V];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = min(r0 + r, a.rows - 1), l = static_cast<int>(a.div_G.div(row)), h = n * a.G + row - l * a.G;
        const T *of = static_cast<const T *>(a.q) + b * a.qs[0] + l * a.qs[1] + h * a.qs[2] + m * a.qs[3];
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            load_row<T, V>(of, (i * 16 + sub) * V, a.D, q[r][i]);
#pragma unroll
            for (int e = 0; e < V; ++e) q[r][i][e] *= a.scale_log2;
        }
    }
    // The lane's score: of key `ki` of a batch with row r0 + ri.
    const int ki = sub / R, ri = sub % R, my_row = min(r0 + ri, a.rows - 1);
    const int my_l = static_cast<int>(a.div_G.div(my_row)), my_h = n * a.G + my_row - my_l * a.G;
    const int my_pos = a.pos_q ? a.pos_q[static_cast<int64_t>(b) * a.Lq + my_l] : old + my_l;
    const bool my_live = ki < KB && r0 + ri < a.rows && my_l < count;
    float top = -FLT_MAX, sum = 0.f;  // of the lane's row and map; its own keys' sum
    float o[R][2][NV][V];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < NV; ++c)
#pragma unroll
                for (int e = 0; e < V; ++e) o[r][i][c][e] = 0.f;

    const T *const kb = static_cast<const T *>(a.k) + n * a.ks[2] + m * a.ks[3], *const vb = static_cast<const T *>(a.v) + n * a.vs[2];
    // 32 keys at a time: a lane finds out where one of them is.
    for (int j0 = jb + warp * 32; j0 < end; j0 += kFewWarps * 32) {
        const int mine = j0 + lane;
        int page = -1, place = 0, pos = mine;
        if (mine < end) {
            const int64_t of = static_cast<int64_t>(b) * a.Lk + mine;
            page = paged_page(a, b, mine, place);
            if (a.mask && !a.mask[of]) page = -1;
            if (a.pos_k) pos = a.pos_k[of];
        }
        const int batches = (min(32, end - j0) + KB - 1) / KB;
#pragma unroll 1
        for (int t = 0; t < batches; ++t) {
            float kt[KB][NK][V], vt[KB][NV][V];
#pragma unroll
            for (int i = 0; i < KB; ++i) {
                const int pg = __shfl_sync(0xffffffffu, page, t * KB + i), pl = __shfl_sync(0xffffffffu, place, t * KB + i);
                const bool there = pg >= 0;
                const T *kr = kb + (there ? pg * a.ks[0] + pl * a.ks[1] : 0), *vr = vb + (there ? pg * a.vs[0] + pl * a.vs[1] : 0);
#pragma unroll
                for (int c = 0; c < NK; ++c) load_row<T, V>(kr, (c * 16 + sub) * V, there ? a.D : 0, kt[i][c]);
#pragma unroll
                for (int c = 0; c < NV; ++c) load_row<T, V>(vr, (c * 32 + lane) * V, there ? a.Dv : 0, vt[i][c]);
            }
            float dots[16];
#pragma unroll
            for (int i = KB * R; i < 16; ++i) dots[i] = 0.f;
#pragma unroll
            for (int i = 0; i < KB; ++i)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float d = 0.f;
#pragma unroll
                    for (int c = 0; c < NK; ++c)
#pragma unroll
                        for (int e = 0; e < V; ++e) d = fmaf(q[r][c][e], kt[i][c][e], d);
                    dots[i * R + r] = d;
                }
            float s = fold16(dots, lane);
            const int from = (t * KB + ki) & 31, j = j0 + t * KB + ki;  // lanes without a key are not live
            const int rel = __shfl_sync(0xffffffffu, pos, from) - my_pos, my_page = __shfl_sync(0xffffffffu, page, from);
            bool see = my_live && my_page >= 0 && !(a.causal && rel > 0);
            if (see && a.pg.tree && j >= old) see = a.pg.tree[(static_cast<int64_t>(b) * a.Lq + my_l) * a.Lq + j - old] != 0;
            if (a.nb) {
                const int bucket = min(max(a.bmap[min(max(rel, -a.reach), a.reach) + a.reach], 0), a.nb - 1);
                s += a.table[bucket * a.H + my_h] * kLog2e;
            }
            s = see ? s : -INFINITY;
            // The row's maximum over the batch's keys, in all of its lanes.
            float best = s;
#pragma unroll
            for (int x = R; x < 16; x <<= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, x));
            if (__any_sync(0xffffffffu, best > top)) {
                const float next = fmaxf(best, top), shrink = ex2(top - next);
                top = next;
                sum *= shrink;
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float f = __shfl_sync(0xffffffffu, shrink, i * 16 + r);
#pragma unroll
                        for (int c = 0; c < NV; ++c)
#pragma unroll
                            for (int e = 0; e < V; ++e) o[r][i][c][e] *= f;
                    }
            }
            const float p = ex2(s - top);
            sum += p;
#pragma unroll
            for (int i = 0; i < KB; ++i)
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float w = __shfl_sync(0xffffffffu, p, x * 16 + i * R + r);
#pragma unroll
                        for (int c = 0; c < NV; ++c)
#pragma unroll
                            for (int e = 0; e < V; ++e) o[r][x][c][e] = fmaf(w, vt[i][c][e], o[r][x][c][e]);
                    }
        }
    }
    // The row's sum over its lanes, then the warps' parts in a fixed order.
#pragma unroll
    for (int x = R; x < 16; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    __shared__ float tops[kFewWarps][2][R], sums[kFewWarps][2][R];
    extern __shared__ float outs[];  // [warps][R][2][Dv]
    if (sub < R) {
        tops[warp][m][sub] = top;
        sums[warp][m][sub] = sum;
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < NV; ++c)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const int d = (c * 32 + lane) * V + e;
                    if (d < a.Dv) outs[((warp * R + r) * 2 + i) * a.Dv + d] = o[r][i][c][e];
                }
    __syncthreads();
    for (int x = threadIdx.x; x < R * a.Dv; x += kFewThreads) {
        const int r = x / a.Dv, d = x - r * a.Dv, row = r0 + r;
        if (row >= a.rows) continue;
        const int l = static_cast<int>(a.div_G.div(row)), h = n * a.G + row - l * a.G;
        float all[2], total[2], most[2];
        for (int i = 0; i < 2; ++i) {
            most[i] = -FLT_MAX;
            for (int w = 0; w < kFewWarps; ++w) most[i] = fmaxf(most[i], tops[w][i][r]);
            all[i] = total[i] = 0.f;
            for (int w = 0; w < kFewWarps; ++w) {
                const float f = ex2(tops[w][i][r] - most[i]);
                total[i] = fmaf(sums[w][i][r], f, total[i]);
                all[i] = fmaf(outs[((w * R + r) * 2 + i) * a.Dv + d], f, all[i]);
            }
            if (total[i] == 0.f) all[i] = 0.f;  // no keys: not even 0 times a value that is not finite
        }
        if (a.splits > 1) {
            const int64_t at = ((static_cast<int64_t>(b) * a.Hkv + n) * a.rows + row) * a.splits + split;
            for (int i = 0; i < 2; ++i) {
                a.part_o[(at * 2 + i) * a.Dv + d] = all[i];
                if (d == 0) {
                    a.part_ml[(at * 2 + i) * 2] = most[i];
                    a.part_ml[(at * 2 + i) * 2 + 1] = total[i];
                }
            }
        } else {
            const float y = total[1] == 0.f ? 0.f : a.lam[h] * (all[1] / total[1]);
            static_cast<T *>(a.out)[((static_cast<int64_t>(b) * a.Lq + l) * a.H + h) * a.Dv + d] =
                dattn_round<T>((total[0] == 0.f ? 0.f : all[0] / total[0]) - y);
        }
    }
}

// Joins the parts of a row that was split over the keys. A warp takes a row, or
// with many parts (WARPS = 8) the block's warps share one.
template <typename T, int WARPS> __global__ void __launch_bounds__(256) paged_merge_kernel(const __grid_constant__ DattnArgs a)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = WARPS == 1 ? 0 : warp;
    const int64_t row = WARPS == 1 ? static_cast<int64_t>(blockIdx.x) * 8 + warp : blockIdx.x;
    const int bn = static_cast<int>(row / a.rows);
    if (bn >= a.B * a.Hkv) return;
    pdl_wait();
    const int r = static_cast<int>(row - static_cast<int64_t>(bn) * a.rows), b = bn / a.Hkv, n = bn - b * a.Hkv;
    const int l = static_cast<int>(a.div_G.div(r)), h = n * a.G + r - l * a.G;
    const auto ml = [&](int i) {  // of both maps
        if (i >= a.splits) return make_float4(-FLT_MAX, 0.f, -FLT_MAX, 0.f);
        const float4 p = *reinterpret_cast<const float4 *>(a.part_ml + (row * a.splits + i) * 4);
        return make_float4(fmaxf(p.x, -FLT_MAX), p.y, fmaxf(p.z, -FLT_MAX), p.w);
    };
    float top[2] = {-FLT_MAX, -FLT_MAX}, sum[2] = {0.f, 0.f};
    for (int i = lane; i < a.splits; i += 32) {
        const float4 x = ml(i);
        top[0] = fmaxf(top[0], x.x);
        top[1] = fmaxf(top[1], x.z);
    }
    for (int m = 0; m < 2; ++m)
        for (int k = 16; k; k >>= 1) top[m] = fmaxf(top[m], __shfl_xor_sync(0xffffffffu, top[m], k));
    // A lane takes channels lane, lane + 32, ..; parts past the last have a factor of 0.
    constexpr int NC = DATTN_MAX_VALUE_WIDTH / 32;
    float o[2][NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) o[0][c] = o[1][c] = 0.f;
    for (int base = part * 4; base < a.splits; base += WARPS * 4) {
        const float4 w = ml(base + (lane & 3));
        const float f[2] = {ex2(w.x - top[0]), ex2(w.z - top[1])};
        if (lane < 4) {
            sum[0] = fmaf(w.y, f[0], sum[0]);
            sum[1] = fmaf(w.w, f[1], sum[1]);
        }
        float x[4][2][NC];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    x[i][m][c] = base + i < a.splits && c * 32 + lane < a.Dv ? a.part_o[((row * a.splits + base + i) * 2 + m) * a.Dv + c * 32 + lane] : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float g = __shfl_sync(0xffffffffu, f[m], i);
#pragma unroll
                for (int c = 0; c < NC; ++c) o[m][c] = fmaf(x[i][m][c], g, o[m][c]);
            }
    }
    for (int m = 0; m < 2; ++m)
        for (int k = 2; k; k >>= 1) sum[m] += __shfl_xor_sync(0xffffffffu, sum[m], k);
    sum[0] = __shfl_sync(0xffffffffu, sum[0], 0);
    sum[1] = __shfl_sync(0xffffffffu, sum[1], 0);
    if constexpr (WARPS > 1) {
        __shared__ float sums[WARPS][2], outs[WARPS][2][NC * 32];
        if (lane < 2) sums[warp][lane] = lane ? sum[1] : sum[0];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int c = 0; c < NC; ++c) outs[warp][m][c * 32 + lane] = o[m][c];
        __syncthreads();
        if (warp > 0) return;
        for (int m = 0; m < 2; ++m) {
            sum[m] = 0.f;
            for (int w = 0; w < WARPS; ++w) sum[m] += sums[w][m];
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                o[m][c] = 0.f;
                for (int w = 0; w < WARPS; ++w) o[m][c] += outs[w][m][c * 32 + lane];
            }
    }
    // Parts of a row without keys are zeros; lam may be anything.
    const float f0 = sum[0] == 0.f ? 0.f : 1.f / sum[0], f1 = sum[1] == 0.f ? 0.f : 1.f / sum[1], lam = sum[1] == 0.f ? 0.f : a.lam[h];
#pragma unroll
    for (int c = 0; c < NC; ++c)
        if (c * 32 + lane < a.Dv)
            static_cast<T *>(a.out)[((static_cast<int64_t>(b) * a.Lq + l) * a.H + h) * a.Dv + c * 32 + lane] =
                dattn_round<T>(o[0][c] * f0 - lam * (o[1][c] * f1));
}

template <typename T> cudaError_t merge(const DattnArgs &a, cudaStream_t st)
{
    const int64_t rows = static_cast<int64_t>(a.B) * a.Hkv * a.rows;
    if (a.splits > 16) return launch_pdl(paged_merge_kernel<T, 8>, dim3(static_cast<unsigned>(rows)), dim3(256), 0, st, a);
    return launch_pdl(paged_merge_kernel<T, 1>, dim3(static_cast<unsigned>((rows + 7) / 8)), dim3(256), 0, st, a);
}

template <typename T, int R, int KB, int V, int NK, int NV> cudaError_t launch_few(const DattnArgs &a, cudaStream_t st)
{
    const size_t row = sizeof(float) * kFewWarps * R * 2;  // of one channel
    const auto kernel = paged_few_kernel<T, R, KB, V, NK, NV>;
    if (const cudaError_t e = allow_shared(kernel, row * NV * 32 * V); e != cudaSuccess) return e;
    kernel<<<dim3(static_cast<unsigned>((a.rows + R - 1) / R * a.splits), a.Hkv, a.B), kFewThreads, row * a.Dv, st>>>(a);
    return cudaGetLastError();
}

// Four elements to a load where alignment allows and widths are multiples of
// four. Up to eight rows stay in registers, two of the widest; more are walked
// for by CTAs of their own.
template <typename T> cudaError_t any_few(const DattnArgs &a, bool quads, cudaStream_t st)
{
    if (!quads) return launch_few<T, 2, 2, 1, 8, 8>(a, st);
    if (a.D > 64 || a.Dv > 128) return launch_few<T, 2, 2, 4, 2, 2>(a, st);
    return a.rows <= 2 ? launch_few<T, 2, 8, 4, 1, 1>(a, st) : a.rows <= 4 ? launch_few<T, 4, 4, 4, 1, 1>(a, st) : launch_few<T, 8, 2, 4, 1, 1>(a, st);
}

}  // namespace

cudaError_t paged_forward_few(const DattnArgs &a, int dtype, bool quads, cudaStream_t st)
{
    return dtype == DA_F32 ? any_few<float>(a, quads, st) : dtype == DA_BF16 ? any_few<__nv_bfloat16>(a, quads, st) : any_few<__half>(a, quads, st);
}

cudaError_t paged_merge(const DattnArgs &a, int dtype, cudaStream_t st)
{
    return dtype == DA_F32 ? merge<float>(a, st) : dtype == DA_BF16 ? merge<__nv_bfloat16>(a, st) : merge<__half>(a, st);
}

}  // namespace da
