// Declarations shared by the translation units of the attention over a paged
// cache (include/paged.h). Nothing here is exported.
#pragma once

#include "dattn_internal.cuh"

namespace da {

constexpr int kPgBias = 6 * 1024;  // bytes of bias that a CTA has room for

// Bytes of the bias table and the map of buckets in shared memory.
inline size_t paged_bias_bytes(int nb, int H, int reach) { return nb ? sizeof(float) * nb * H + sizeof(uint16_t) * (2 * reach + 1) : 0; }

struct PagedTcArgs {
    DattnArgs d;        // part_o [2 ctas, RT, 2, Dv], part_ml [2 ctas, RT, 2, 2]
    int32_t *slots;     // [ctas, 2, 2] tile of a slot (-1: none), whether the piece ends it
    int32_t RT;         // rows of a tile: 16, 32 or 64
    int32_t LP;         // queries of a tile
    int32_t row_tiles;  // tiles of a sequence and key head
    int32_t box;        // places that one copy brings
    int32_t ctas;
};

da_status paged_forward_bf16(const PagedTcArgs &a, cudaStream_t st);
da_status paged_forward_f16(const PagedTcArgs &a, cudaStream_t st);

// On the fp32 units: few rows (quads: four elements to a load), and the join of
// rows that were split over the keys.
cudaError_t paged_forward_few(const DattnArgs &a, int dtype, bool quads, cudaStream_t st);
cudaError_t paged_merge(const DattnArgs &a, int dtype, cudaStream_t st);

}  // namespace da
