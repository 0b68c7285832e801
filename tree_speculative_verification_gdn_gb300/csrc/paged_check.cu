#include "paged_check.cuh"
#include "tv_launch.cuh"

namespace tv {
namespace {

__global__ void __launch_bounds__(256) paged_check_kernel(PagedCheck c, int32_t* __restrict__ err) {
  plan_begun();
  int n;
  const int st = check_sequence(c, blockIdx.x, n);
  if (threadIdx.x == 0) err[blockIdx.x] = st;
}

}  // namespace

cudaError_t launch_paged_check(const PagedCheck& c, int32_t* err, cudaStream_t s) {
  paged_check_kernel<<<c.B, 256, 0, s>>>(c, err);
  return cudaGetLastError();
}

}  // namespace tv
