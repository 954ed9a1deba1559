// hhr_paged_attend: fp16 queries, the same type of cache.
#include "paged_attend.cuh"

namespace hhr {
cudaError_t launch_paged_f16(const PagedArgs& a, int d, int grid, cudaStream_t s) {
  return launch_paged_typed<__half, __half>(a, d, grid, s);
}
}  // namespace hhr
