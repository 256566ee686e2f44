/*
 * dattn.h: differential attention with a learned relative position bias by
 * buckets (C ABI of libda.so).
 *
 * Sequences of Lq queries and Lk keys per batch item, H query heads, Hkv key
 * heads (H % Hkv == 0; query head h reads key head h / (H / Hkv)). Each head
 * has two query and two key vectors of width D and one value of width Dv:
 *
 *   t_m[i,j] = scale * q[i,h,m] . k[j,h',m] + bias[i,j,h]         m = 0, 1
 *   bias     = bias_table[bucket_map[clamp(r, -reach, reach) + reach], h]
 *   r        = pos_k[j] - pos_q[i]
 *   P_m[i,:] = softmax of t_m[i,:] over the keys that query i sees
 *   out[i,h] = sum_j (P_0[i,j] - lam[h] * P_1[i,j]) * v[j,h']
 *
 * Query i sees key j when j < key_lengths[b], key_mask[b,j] != 0 and, if
 * causal, r <= 0. A query that sees no key gets out = 0 and gives no
 * gradient. What q holds for such a query, and k and v for a key that
 * key_lengths or key_mask excludes, is not used: NaN or infinity there
 * reaches no result.
 * A bias of -infinity hides its bucket's keys in the same way, and so does one
 * whose product with log2(e) is not finite, such as the lowest finite value: a
 * query that sees no other key gets 0. Other biases and scores may have any
 * size; a weight is good to 2^-24 times the size of its score.
 *
 * Without pos_k, key j is at position j; without pos_q, query i is at
 * key_lengths[b] - Lq + i (the queries are the last of the sequence), with
 * Lk for key_lengths[b] where that is absent.
 *
 * With g = grad_out and P = P_0 - lam * P_1, the backward pass is
 *   e[i,j] = g[i] . v[j],   d_m[i] = sum_j P_m[i,j] e[i,j]
 *   s_0 = P_0 * (e - d_0),  s_1 = -lam * P_1 * (e - d_1)
 *   grad_v[j] = sum_i P[i,j] g[i]               over the query heads that
 *   grad_k[j,m] = scale * sum_i s_m[i,j] q[i,m] share the key head
 *   grad_q[i,m] = scale * sum_j s_m[i,j] k[j,m]
 *   grad_lam[h] = -sum_i d_1[i]
 *   grad_table[n,h] = sum of s_0 + s_1 over the (b, i, j) of bucket n
 *
 * Conventions are those of da.h (device/host pointers, stream, validation,
 * da_last_error). Scores, softmax statistics and every sum are fp32. bf16 and
 * fp16 inputs go through the tensor cores where dattn_path() says so; there
 * the weights P, and s_m in the backward pass, are rounded to the inputs'
 * type as operands of the second products, as the tensor cores require.
 * grad_lam and grad_table are formed from the unrounded values.
 * In fp16 these operands have powers of two of their own, by bounds of lam,
 * grad_out and v, that bring them into the type's range and are taken out of
 * the sums: only the gradients themselves, as values of that type, are to be
 * scaled as fp16 training does.
 * Sums are taken in a fixed order: results do not vary from run to run.
 * Positions lie in (-2^30, 2^30). Device-side indices are bounded in every
 * build: key_lengths is clamped to [0, Lk] and bucket_map to the table.
 */
#ifndef DATTN_H_
#define DATTN_H_

#include "da.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DATTN_MAX_WIDTH 128        /* largest D */
#define DATTN_MAX_VALUE_WIDTH 256  /* largest Dv */
#define DATTN_MAX_REACH 1024       /* largest reach */
#define DATTN_MAX_TABLE 512        /* largest num_buckets * H / Hkv */

typedef struct dattn_problem {
    int32_t batch;        /* B >= 0 */
    int32_t num_queries;  /* Lq >= 0 */
    int32_t num_keys;     /* Lk >= 0 */
    int32_t num_heads;    /* H >= 1 */
    int32_t num_kv_heads; /* Hkv >= 1, H % Hkv == 0 */
    int32_t width;        /* D, 1..DATTN_MAX_WIDTH */
    int32_t value_width;  /* Dv, 1..DATTN_MAX_VALUE_WIDTH */
    int32_t dtype;        /* a da_dtype: of q, k, v, out and their gradients */
    int32_t num_buckets;  /* 0: no bias */
    int32_t reach;        /* >= 1 with a bias */
    int32_t causal;       /* 0 or 1 */
    float scale;          /* finite */
    /* Device tensors [B, Lq, H, 2, D], [B, Lk, Hkv, 2, D], [B, Lk, Hkv, Dv];
     * the last dimension contiguous, the others' strides in elements: batch,
     * position, head and (q, k) map. Strides are >= 0. Aligned to elements. */
    const void *q, *k, *v;
    int64_t q_stride[4], k_stride[4], v_stride[3];
    const float *lam;            /* device [H] fp32 */
    const float *bias_table;     /* device [num_buckets, H] fp32, or NULL */
    const int32_t *bucket_map;   /* device [2*reach + 1] int32, or NULL */
    const int32_t *pos_q;        /* device [B, Lq] int32, or NULL */
    const int32_t *pos_k;        /* device [B, Lk] int32, or NULL */
    const uint8_t *key_mask;     /* device [B, Lk], 0 or 1, or NULL */
    const int32_t *key_lengths;  /* device [B] int32, or NULL */
} dattn_problem;

/* Which kernels dattn_forward (backward == 0) or dattn_backward takes (a
 * host-only rule on types, sizes and alignment): 1 the tensor-core ones, 0 the
 * general ones, < 0 invalid. */
int32_t dattn_path(const dattn_problem *p, int32_t backward);

/* Bytes of device scratch of dattn_forward (backward == 0) or dattn_backward. */
da_status dattn_workspace_size(const dattn_problem *p, int32_t backward, size_t *bytes);

/*
 * dattn_forward
 *   out   device [B, Lq, H, Dv], dtype, contiguous; overwritten.
 *   out1  device [B, Lq, H, n, Dv], dtype, contiguous, and
 *   lse   device [B, H, 2, Lq] fp32: what dattn_backward needs besides out.
 *         fp32: n = 1, the second map's own output sum_j P_1 v. bf16 and fp16:
 *         n = 3, what rounding took from out, the second map's own output, and
 *         what rounding took from that (both rests times 2^11 in fp16).
 *         lse is the log2 of both maps' sums of 2^(t*log2 e), +infinity where
 *         a query sees no key. Both NULL, or neither.
 *   workspace  device, 256-byte aligned.
 */
da_status dattn_forward(const dattn_problem *p, void *out, void *out1, float *lse, void *workspace,
                        size_t workspace_bytes, da_stream_t stream);

/*
 * dattn_backward: p as given to dattn_forward; out, out1, lse as it wrote them.
 *   grad_out  device, like out.
 *   grad_q, grad_k, grad_v  device, contiguous, of q's, k's and v's shapes.
 *   grad_lam  device [H] fp32.
 *   grad_table  device [num_buckets, H] fp32; NULL without a bias.
 */
da_status dattn_backward(const dattn_problem *p, const void *out, const void *out1, const float *lse,
                         const void *grad_out, void *grad_q, void *grad_k, void *grad_v, float *grad_lam,
                         float *grad_table, void *workspace, size_t workspace_bytes, da_stream_t stream);

/*
 * The kernels' waits on their own copies and products end after a bounded
 * number of tries. A wait that ran out (none does in a sound run) sets a word
 * on the device and turns the call's outputs into NaN. This call waits for
 * `stream`, reads the word into *gave_up (host) and clears it.
 */
da_status dattn_device_status(uint32_t *gave_up, da_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DATTN_H_ */
