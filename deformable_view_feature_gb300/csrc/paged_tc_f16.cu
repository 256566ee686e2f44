// The attention over a paged cache on the tensor cores, for f16: a translation
// unit of its own for each type, because they take long to compile.
#include "paged_tc.cuh"

namespace da {

da_status paged_forward_f16(const PagedTcArgs &a, cudaStream_t st) { return forward_tensor<__half>(a, DA_F16, st); }
uint32_t *paged_gave_up_f16() { return gave_up_word(); }

}  // namespace da
