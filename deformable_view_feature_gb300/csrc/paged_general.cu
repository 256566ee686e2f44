// Differential attention over a paged cache (include/paged.h) on the fp32 units,
// in tiles: the forward kernel of dattn_general.cuh with rows fetched by page.
#include "dattn_general.cuh"

namespace da {
namespace {

template <typename T> cudaError_t paged_width(const DattnArgs &a, cudaStream_t st)
{
    switch (padded_width(a)) {
    case 32: return forward_width<T, 32, true>(a, st);
    case 64: return forward_width<T, 64, true>(a, st);
    default: return forward_width<T, 128, true>(a, st);
    }
}

}  // namespace

cudaError_t paged_forward_general(const DattnArgs &a, int dtype, cudaStream_t st)
{
    switch (dtype) {
    case DA_F32: return paged_width<float>(a, st);
    case DA_BF16: return paged_width<__nv_bfloat16>(a, st);
    default: return paged_width<__half>(a, st);
    }
}

}  // namespace da
