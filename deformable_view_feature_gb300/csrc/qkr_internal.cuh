// Declarations shared by the rotary norm (qkr.h) and the paged append
// (paged.h). Nothing here is exported.
#pragma once

#include "da_internal.cuh"
#include "paged.h"

namespace da {

// One tensor of vectors, [B, L, H, M, D]: queries, keys, or values that are
// copied (M = 1, R = 0, not normed).
//
// Lanes and channels: a lane owns a slot of a vector, two pieces of V channels,
// so that both halves of a rotated pair are in one lane's registers and a pass
// exchanges nothing but the sum of squares. The first nr slots hold the rotated
// channels (pieces at t*V and R/2 + t*V, or neighbours where interleaved), the
// others two neighbouring pieces of the rest.
struct QkrSide {
    const void *x, *g;   // inputs; backward: and the outputs' gradients
    void *y;             // outputs; backward: the inputs' gradients
    int64_t xs[4];       // strides of x: batch, position, head, map
    int64_t ys[4];       // of y, and of g; paged: page, place, head, map
    const float *w;
    const int32_t *pos;
    int32_t L, H, M, D, R;
    int32_t first;       // position of token 0 without pos
    int32_t nr, slots, sg_log2;  // slots that rotate, slots, log2 of the lanes of a vector
    int32_t tpw;         // tokens that a warp takes at once
    int32_t parts, per;  // forward: warps that share a token, vectors of each
    int32_t paged, normed, keys;
    float inv_D;         // 1 / D
    int64_t tokens;      // B * L
    int64_t unit0;       // its first CTA
    int32_t units;       // its CTAs
    FastDiv div_L, div_vec, div_hp;  // by L, H * M, R / 2
    float *grad_w, *part;            // backward: [D], and [units, D]
};

struct QkrArgs {
    QkrSide side[3];
    int32_t sides;
    int32_t interleaved;
    const int64_t *turns;
    float eps, magnitude;
    // Of a paged side.
    const int32_t *table, *lengths, *counts;
    int32_t table_pages, page_size, num_pages;
    FastDiv div_page;
};

// Checks p and fills the sides of queries and keys that there are (with their
// inputs, and outputs y of contiguous layout).
da_status qkr_sides(const qkr_problem *p, const void *out_q, const void *out_k, QkrArgs &a);
da_status qkr_launch_forward(QkrArgs &a, int dtype, cudaStream_t st);

}  // namespace da
