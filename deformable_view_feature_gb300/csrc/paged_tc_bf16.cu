// The attention over a paged cache on the tensor cores, for bf16: a translation
// unit of its own for each type, because they take long to compile.
#include "paged_tc.cuh"

namespace da {

da_status paged_forward_bf16(const PagedTcArgs &a, cudaStream_t st) { return forward_tensor<__nv_bfloat16>(a, DA_BF16, st); }
uint32_t *paged_gave_up_bf16() { return gave_up_word(); }

}  // namespace da
