// hhr_paged_attend: fp16 queries, 8-bit cache.
#include "paged_attend.cuh"

namespace hhr {
cudaError_t launch_paged_f16_e4m3(const PagedArgs& a, int d, int grid, cudaStream_t s) {
  return launch_paged_typed<__half, __nv_fp8_e4m3>(a, d, grid, s);
}
}  // namespace hhr
