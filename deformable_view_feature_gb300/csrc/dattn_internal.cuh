// Declarations shared by the differential-attention translation units
// (include/dattn.h). Nothing here is exported.
#pragma once

#include <cuda_bf16.h>

#include "da_internal.cuh"
#include "dattn.h"

namespace da {

// The problem as the kernels see it. The G = H / Hkv query heads that share a
// key head are handled together: a "row" is one (query, head) pair, row r of
// key head n being query r / G of head n*G + r % G. One token of a serving
// batch thus still fills a tile with its G heads, and keys are read once for
// all of them.
struct DattnArgs {
    const void *q, *k, *v;
    int64_t qs[4], ks[4], vs[3];
    const float *lam, *table;
    const int32_t *bmap, *pos_q, *pos_k, *lengths;
    const uint8_t *mask;
    int32_t B, Lq, Lk, H, Hkv, G, D, Dv, nb, reach, causal;
    int32_t wide;       // fp32, widths and strides of whole 16 bytes, aligned
    int32_t rows;       // Lq * G
    FastDiv div_G;
    float scale;        // of the scores
    float scale_log2;   // scale * log2(e): scores are kept times log2(e)
    void *out, *out1;   // forward outputs (backward: inputs); out1 [B, Lq, H, kSaved, Dv]
    float *lse;         // [B, H, 2, Lq]
    // Forward split over the keys: `splits` CTAs share a tile of rows, each
    // leaving its unnormalised sums [.., 2, Dv], and maximum and sum [.., 2, 2].
    int32_t splits, keys_per_split;
    float *part_o, *part_ml;
    // Backward.
    const void *grad_out;
    void *grad_q, *grad_k, *grad_v;
    float *grad_lam, *grad_table;
    float *delta;       // [B, Hkv, 2, rows] the d_m of dattn.h
    uint32_t *most;     // fp16 on the tensor cores: [2, B * Hkv] bits of the largest |v| and bound of grad_out
    float *part_table;  // [key-tile CTAs, nb * G]
    int32_t table_ctas; // CTAs of the second kernel per (b, key head)
    // The general kernels' splits backward: grad_q over the keys (splits,
    // keys_per_split, part_o [.., 2, D], part_ml [.., 2]), grad_k and grad_v
    // over the rows (part_kv [.., Dv + 2 D]).
    int32_t row_splits;
    int32_t own_sums;   // bucket sums of every thread, not of every warp
    float *part_kv;
};

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ int dattn_length(const DattnArgs &a, int b)
{
    return a.lengths ? min(max(a.lengths[b], 0), a.Lk) : a.Lk;
}

template <typename T> __device__ __forceinline__ float dattn_float(T v);
template <> __device__ __forceinline__ float dattn_float(float v) { return v; }
template <> __device__ __forceinline__ float dattn_float(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float dattn_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T dattn_round(float v);
template <> __device__ __forceinline__ float dattn_round(float v) { return v; }
template <> __device__ __forceinline__ __half dattn_round(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 dattn_round(float v) { return __float2bfloat16_rn(v); }

// What the backward pass needs of the outputs, kSaved<T> words for each value:
// map 1's own output, and in 16 bits also what rounding took from out, before
// it, and from map 1's, after it. The d_m of dattn.h are sums over g times the
// outputs; from rounded ones their error, times the mean key, is the largest
// of grad_q wherever keys have a common part. Two words hold 16 bits of a bf16
// output and 22 of an fp16 one, whose second word is scaled to stay normal.
template <typename T> constexpr int kSaved = sizeof(T) == 2 ? 3 : 1;
template <typename T> constexpr float kRest = 1.f;
template <> constexpr float kRest<__half> = 2048.f;
template <typename T> __device__ __forceinline__ T dattn_rest(float v, T rounded)
{
    return dattn_round<T>((v - dattn_float(rounded)) * kRest<T>);
}
template <typename T> __device__ __forceinline__ float dattn_whole(T rounded, T rest)
{
    return fmaf(dattn_float(rest), 1.f / kRest<T>, dattn_float(rounded));
}

// Stores value d of an output and of map 1's own, and what is saved of them
// (out1 may be null).
template <typename T> __device__ __forceinline__ void dattn_store(const DattnArgs &a, int64_t row, int d, float out, float own1)
{
    const T u = dattn_round<T>(out);
    static_cast<T *>(a.out)[row * a.Dv + d] = u;
    if (!a.out1) return;
    T *save = static_cast<T *>(a.out1) + row * kSaved<T> * a.Dv + d;
    const T w = dattn_round<T>(own1);
    if constexpr (sizeof(T) == 2) {
        save[0] = dattn_rest(out, u);
        save[a.Dv] = w;
        save[2 * a.Dv] = dattn_rest(own1, w);
    } else {
        save[0] = w;
    }
}

da_status dattn_forward_tensor(const DattnArgs &a, int dtype, cudaStream_t st);
da_status dattn_backward_tensor(const DattnArgs &a, int dtype, cudaStream_t st);
uint32_t *dattn_gave_up_word();           // of the forward kernels
uint32_t *dattn_gave_up_backward_word();  // of the backward kernels
cudaError_t dattn_forward_general(const DattnArgs &a, int dtype, cudaStream_t st);
cudaError_t dattn_backward_general(const DattnArgs &a, int dtype, cudaStream_t st);
cudaError_t dattn_merge(const DattnArgs &a, int dtype, cudaStream_t st);
cudaError_t dattn_finish_backward(const DattnArgs &a, cudaStream_t st);
int dattn_general_row_tile(const DattnArgs &a);   // rows of a forward tile
int dattn_general_tile(const DattnArgs &a);       // rows, and keys, of a backward tile

}  // namespace da
