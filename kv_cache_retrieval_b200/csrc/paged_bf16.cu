// hhr_paged_attend: bf16 queries, the same type of cache.
#include "paged_attend.cuh"

namespace hhr {
cudaError_t launch_paged_bf16(const PagedArgs& a, int d, int grid, cudaStream_t s) {
  return launch_paged_typed<__nv_bfloat16, __nv_bfloat16>(a, d, grid, s);
}
}  // namespace hhr
