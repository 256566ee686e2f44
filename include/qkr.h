/*
 * qkr.h: norm of every head's queries and keys and their rotation by position
 * (C ABI of libda.so).
 *
 * The queries and keys are those of the differential attention (dattn.h):
 * q [B, Lq, H, 2, D] and k [B, Lk, Hkv, 2, D], two vectors of width D per
 * head. Each vector x on its own becomes z:
 *
 *   n = x / sqrt(mean(x^2) + eps),  y = weight * n        (normed; else y = x)
 *   of the first R = rotated channels, in pairs (a, b):
 *     z_a = magnitude * (y_a cos t - y_b sin t)
 *     z_b = magnitude * (y_a sin t + y_b cos t),  t = 2 pi * pos * turns[i] / 2^64
 *   the channels from R on: z = y
 *
 * Pair i is (i, R/2 + i), or (2 i, 2 i + 1) where interleaved. turns[i] is the
 * pair's angle for one position in units of 2^-64 of a turn, as a signed 64-bit
 * number, so that the product with any 32-bit position, taken modulo 2^64, is
 * exact: far positions lose no digits.
 *
 * With g the gradient of z, turned back by the same angle (g_y), the backward
 * pass is
 *   grad_weight = sum g_y * n                        over all the tensor's vectors
 *   grad_x = (weight*g_y - n * mean(weight*g_y*n)) / sqrt(mean(x^2) + eps)
 *
 * Conventions are those of da.h (device/host pointers, stream, validation,
 * da_last_error). Arithmetic is fp32, results are rounded once to the tensors'
 * type. Sums are taken in a fixed order: results do not vary from run to run.
 * Bounds-checking builds: the kernels here compute no index from device data.
 */
#ifndef QKR_H_
#define QKR_H_

#include "da.h"

#ifdef __cplusplus
extern "C" {
#endif

#define QKR_MAX_WIDTH 128 /* largest D */

typedef struct qkr_problem {
    int32_t batch;        /* B >= 0 */
    int32_t num_queries;  /* Lq >= 0; 0: no queries */
    int32_t num_keys;     /* Lk >= 0; 0: no keys */
    int32_t num_heads;    /* H >= 1 */
    int32_t num_kv_heads; /* Hkv >= 1 */
    int32_t width;        /* D, 1..QKR_MAX_WIDTH */
    int32_t rotated;      /* R, even, 0..D; 0: no rotation */
    int32_t dtype;        /* a da_dtype: of q, k, outputs and gradients */
    int32_t interleaved;  /* 0 or 1 */
    int32_t normed;       /* 0 or 1 */
    float eps;            /* > 0, finite, where normed */
    float magnitude;      /* finite */
    /* Device tensors; the last dimension contiguous, the others' strides in
     * elements: batch, position, head and map. Strides are >= 0. Aligned to
     * elements. */
    const void *q, *k;
    int64_t q_stride[4], k_stride[4];
    const float *q_weight, *k_weight; /* device [D] fp32, or NULL: 1 */
    const int64_t *turns;             /* device [R/2]; may be NULL where R = 0 */
    const int32_t *pos_q;             /* device [B, Lq], or NULL: Lk - Lq + i (i without keys), the last of the sequence */
    const int32_t *pos_k;             /* device [B, Lk], or NULL: j */
} qkr_problem;

/*
 * qkr_forward
 *   out_q, out_k  device [B, Lq, H, 2, D] and [B, Lk, Hkv, 2, D], dtype,
 *                 contiguous; overwritten. Each may be its input where that is
 *                 contiguous; otherwise they overlap no input.
 */
da_status qkr_forward(const qkr_problem *p, void *out_q, void *out_k, da_stream_t stream);

/* Bytes of device scratch of qkr_backward; host-only. */
da_status qkr_workspace_size(const qkr_problem *p, size_t *bytes);

/*
 * qkr_backward: p as given to qkr_forward (q and k as they were before it).
 *   grad_out_q, grad_out_k  device, contiguous, like out_q and out_k.
 *   grad_q, grad_k          device, contiguous; overwritten. Each may be its
 *                           grad_out.
 *   grad_q_weight, grad_k_weight  device [D] fp32; overwritten. NULL exactly
 *                           where the weight is. Zeros where there is no vector.
 *   workspace               device, 256-byte aligned.
 */
da_status qkr_backward(const qkr_problem *p, const void *grad_out_q, const void *grad_out_k, void *grad_q, void *grad_k,
                       float *grad_q_weight, float *grad_k_weight, void *workspace, size_t workspace_bytes,
                       da_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QKR_H_ */
