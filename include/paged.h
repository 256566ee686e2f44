/*
 * paged.h: a cache of keys and values in pages, the step that stores new
 * tokens into it, and differential attention over it (C ABI of libda.so).
 *
 * The cache holds the history of B sequences: keys [P, S, Hkv, 2, D] and values
 * [P, S, Hkv, Dv], P pages of S places each. page_table [B, N] gives each
 * sequence's pages in order: place j of sequence b is place j % S of page
 * page_table[b, j / S], 0 <= j < N * S. Sequences may share pages that are only
 * read. Entries that no token reaches may hold anything; a page number outside
 * [0, P) holds no place: nothing is written there, and its keys are not seen.
 *
 * New tokens are padded to T per sequence; sequence b has counts[b] of them
 * (clamped to [0, T]; T without counts), the first ones of its row.
 *
 * Conventions are those of da.h (device/host pointers, stream, validation,
 * da_last_error). Device-side indices are bounded in every build, so no value
 * in page_table, lengths or counts makes a kernel leave its tensors.
 */
#ifndef PAGED_H_
#define PAGED_H_

#include "dattn.h"
#include "qkr.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct pg_cache {
    /* Device tensors; the last dimension contiguous, the others' strides in
     * elements: page, place, head and (k) map. Strides are >= 0, aligned to
     * elements. Places of one cache may not overlap. */
    void *k, *v;
    int64_t k_stride[4], v_stride[3];
    int32_t num_pages;           /* P >= 0 */
    int32_t page_size;           /* S >= 1 */
    int32_t table_pages;         /* N >= 0, N * S < 2^29 */
    const int32_t *page_table;   /* device [B, N] */
    const int32_t *lengths;      /* device [B]: tokens in the cache */
    const int32_t *counts;       /* device [B], or NULL */
} pg_cache;

/*
 * pg_append: stores new tokens. Token t < counts[b] of sequence b goes to place
 * lengths[b] + t: its keys as qkr.h's z, its values as they are. Its queries
 * become out_q, those of all T tokens, in the same launch.
 *   p       the new tokens: q [B, T, H, 2, D] and k [B, T, Hkv, 2, D] with
 *           num_keys = T and num_queries = T, or 0 without queries. pos_q and
 *           pos_k default to lengths[b] + t.
 *   v       device [B, T, Hkv, value_width], the last dimension contiguous;
 *           v_stride: batch, token, head. value_width is 1..DATTN_MAX_VALUE_WIDTH.
 *   cache   of dtype p->dtype; lengths are those before the call, and are left
 *           as they are. Tokens whose place is outside the table (also at a
 *           length below 0) are not stored; all else in the cache keeps its value.
 *   out_q   device [B, T, H, 2, D], contiguous; may be q where that is
 *           contiguous. NULL without queries.
 * Where two tokens' places coincide (a page in two of a call's written ranges)
 * the place holds an unspecified mixture of the two.
 */
da_status pg_append(const qkr_problem *p, const void *v, const int64_t *v_stride, int32_t value_width,
                    const pg_cache *cache, void *out_q, da_stream_t stream);

/*
 * Attention of the new tokens over the cache: dattn.h's formulas with key j of
 * sequence b at place j, N * S for Lk, and lengths (clamped to [0, N * S]) for
 * key_lengths: what was there before and the new tokens, whose own places are
 * the last counts[b]. By default query i is at position
 * lengths[b] - counts[b] + i and key j at j. Positions lie in (-2^30, 2^30).
 *
 * Query i < counts[b] sees key j when j < lengths[b], its page is in the cache,
 * key_mask[b, j] != 0, and
 *   without tree: if causal, pos_k - pos_q <= 0;
 *   with tree [B, T, T]: j is before the new tokens, or new token
 *   j' = j - (lengths[b] - counts[b]) has tree[b, i, j'] != 0. causal is not
 *   looked at.
 * A query that sees no key, and one with i >= counts[b], gets 0, whatever the
 * cache and lam hold. What the cache holds at places that no query may see (by
 * length, mask or page) is not used: NaN or infinity there reaches no result.
 * (A value that is not finite at a place that some query sees may reach other
 * queries of the sequence, which weigh it with 0, but none that sees no key.)
 * Biases hide keys as in dattn.h.
 *
 * Scores, softmax statistics and sums are fp32. On the tensor cores (bf16, fp16;
 * pg_path) the weights are operands in the inputs' type; up to 64 rows (T * H / Hkv)
 * of groups of up to 32 heads carry what that rounding took as a second operand,
 * more do not. Sums are taken in an order that lengths and counts fix: results do
 * not vary from run to run.
 */
typedef struct pg_problem {
    int32_t batch;        /* B >= 0 */
    int32_t num_tokens;   /* T >= 0 */
    int32_t num_heads;    /* H >= 1 */
    int32_t num_kv_heads; /* Hkv >= 1, H % Hkv == 0 */
    int32_t width;        /* D, 1..DATTN_MAX_WIDTH */
    int32_t value_width;  /* Dv, 1..DATTN_MAX_VALUE_WIDTH */
    int32_t dtype;        /* a da_dtype: of q, the cache and out */
    int32_t num_buckets;  /* 0: no bias */
    int32_t reach;        /* >= 1 with a bias */
    int32_t causal;       /* 0 or 1 */
    float scale;          /* finite */
    const void *q;        /* device [B, T, H, 2, D], strides as in dattn_problem */
    int64_t q_stride[4];
    pg_cache cache;
    const float *lam;           /* device [H] fp32 */
    const float *bias_table;    /* device [num_buckets, H] fp32, or NULL */
    const int32_t *bucket_map;  /* device [2*reach + 1] int32, or NULL */
    const int32_t *pos_q;       /* device [B, T] int32, or NULL */
    const int32_t *pos_k;       /* device [B, N * S] int32, or NULL */
    const uint8_t *key_mask;    /* device [B, N * S], 0 or 1, or NULL */
    const uint8_t *tree;        /* device [B, T, T], 0 or 1, or NULL */
} pg_problem;

/* Which kernels pg_attention takes (a host-only rule on types, sizes and
 * alignment): 1 the tensor-core ones, 0 the general ones, < 0 invalid. The
 * tensor cores take bf16 and fp16 with D and Dv multiples of 8 up to 64 and 128,
 * up to 64 heads to a key head, a page_size that is a multiple of 8, up to 6,144
 * bytes of bias (4 * num_buckets * H + 2 * (2 * reach + 1)), and addresses and
 * strides that are multiples of 16 bytes, none of the strides zero. */
int32_t pg_path(const pg_problem *p);

/* Bytes of device scratch of pg_attention; host-only. */
da_status pg_workspace_size(const pg_problem *p, size_t *bytes);

/*
 * pg_attention
 *   out        device [B, T, H, Dv], dtype, contiguous; overwritten.
 * Its kernels' bounded waits are dattn.h's: dattn_device_status reads them too.
 *   workspace  device, 256-byte aligned.
 */
da_status pg_attention(const pg_problem *p, void *out, void *workspace, size_t workspace_bytes, da_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_H_ */
