// hhr_paged_attend: bf16 queries, 8-bit cache.
#include "paged_attend.cuh"

namespace hhr {
cudaError_t launch_paged_bf16_e4m3(const PagedArgs& a, int d, int grid, cudaStream_t s) {
  return launch_paged_typed<__nv_bfloat16, __nv_fp8_e4m3>(a, d, grid, s);
}
}  // namespace hhr
