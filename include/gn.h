/*
 * gn.h: group norm with an activation over packed channels-last feature maps
 * (C ABI of libda.so).
 *
 * The features are those the deformable aggregation samples (da.h):
 * [B, num_feat_rows, C], one row per pixel, map (k, s) starting at row
 * level_start_index[k, s]. Every map (b, k, s) is normalised on its own, in G
 * groups of C / G consecutive channels:
 *
 *   mean, var = over the H*W pixels and C/G channels of (b, k, s, g)
 *   n = (x - mean) / sqrt(var + eps)      var without Bessel's correction
 *   z = gamma[s, c] * n + beta[s, c]      (or gamma[c], beta[c])
 *   out = act(z)                          z, max(z, 0) or z / (1 + exp(-z))
 *
 * and with h = grad_out * act'(z), the backward pass is
 *
 *   grad_gamma = sum h * n, grad_beta = sum h      over the maps that share it
 *   grad_feat = (gamma*h - mean(gamma*h) - n * mean(gamma*h*n)) / sqrt(var + eps)
 *
 * A plain [B, H, W, C] tensor is the case of one camera and one scale.
 *
 * Conventions are those of da.h (device/host pointers, stream, validation,
 * da_last_error). All arithmetic is fp32: statistics are combined from
 * per-tile means and sums of squared deviations, never from sums of squares
 * about zero. Sums are taken in a fixed order, so results do not vary from
 * run to run. The derivative of max(z, 0) at z = 0 is 0.
 * Bounds-checking builds: the kernels here compute no index from device data.
 */
#ifndef GN_H_
#define GN_H_

#include "da.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gn_act { GN_ACT_NONE = 0, GN_ACT_RELU = 1, GN_ACT_SILU = 2 } gn_act;

#define GN_MAX_CHANNELS 4096

typedef struct gn_dims {
    int32_t batch;         /* B >= 0 */
    int32_t num_cams;      /* K >= 0 */
    int32_t num_scales;    /* S >= 0; K*S <= DA_MAX_MAPS */
    int32_t num_embeds;    /* C, 1..GN_MAX_CHANNELS */
    int32_t num_groups;    /* G >= 1, C % G == 0 */
    int32_t feat_dtype;    /* a da_dtype: of feat, out, grad_out and grad_feat */
    int32_t act;           /* a gn_act */
    int32_t affine_scales; /* 0: gamma, beta are [C]; 1: [S, C] */
    int64_t num_feat_rows; /* rows per batch item, 0 <= rows <= DA_MAX_ROWS */
    float eps;             /* > 0, finite */
} gn_dims;

/* Bytes of device scratch that gn_forward (backward == 0) or gn_backward
 * needs; host-only. */
da_status gn_workspace_size(const gn_dims *dims, const int32_t *spatial_shape, const int32_t *level_start_index,
                            int32_t backward, size_t *bytes);

/*
 * gn_forward
 *   feat              device [B, num_feat_rows, C], feat_dtype, aligned to its
 *                     elements. Rows of C*sizeof(element) = a multiple of 16
 *                     bytes at a 16-byte aligned address take 16-byte accesses.
 *   spatial_shape     host [K, S, 2] int32 and
 *   level_start_index host [K, S] int32, as in da_forward, but the maps may
 *                     not overlap.
 *   gamma, beta       device [C] or [S, C] fp32.
 *   out               device, like feat; overwritten. Rows of no map get 0. It
 *                     may be feat itself.
 *   stats             device [B, K, S, G, 2] fp32, 8-byte aligned: mean and
 *                     1/sqrt(var + eps); overwritten. gn_backward reads it.
 *   workspace         device, 256-byte aligned, gn_workspace_size bytes.
 */
da_status gn_forward(const gn_dims *dims, const void *feat, const int32_t *spatial_shape,
                     const int32_t *level_start_index, const float *gamma, const float *beta, void *out, float *stats,
                     void *workspace, size_t workspace_bytes, da_stream_t stream);

/*
 * gn_backward: feat, gamma, beta as given to gn_forward, stats as it wrote it.
 *   grad_out   device, like feat.
 *   grad_feat  device, like feat; overwritten; rows of no map get 0. It may be
 *              grad_out itself.
 *   grad_gamma, grad_beta  device, fp32, like gamma; overwritten.
 */
da_status gn_backward(const gn_dims *dims, const void *feat, const int32_t *spatial_shape,
                      const int32_t *level_start_index, const float *gamma, const float *beta, const float *stats,
                      const void *grad_out, void *grad_feat, float *grad_gamma, float *grad_beta, void *workspace,
                      size_t workspace_bytes, da_stream_t stream);

/*
 * Tiles whose outputs wait for their map's statistics stop waiting after a
 * bounded number of tries (this happens in no sound run). That sets a word on
 * the device and turns what depended on the wait into NaN: the tiles' outputs,
 * the map's stats, grad_gamma and grad_beta. This call waits for `stream`,
 * reads the word into *gave_up (host) and clears it.
 */
da_status gn_device_status(uint32_t *gave_up, da_stream_t stream);

/*
 * Sets how many tries a wait of later calls, of the whole process, has, and
 * returns the former number; a negative one only returns it. With 0 every wait
 * gives up at once, which is how the way out of a wait is tested.
 */
int32_t da_gn_wait_tries(int32_t tries);

#ifdef __cplusplus
}
#endif

#endif /* GN_H_ */
