#include "paged_check.cuh"
#include "tv_launch.cuh"

namespace tv {
namespace {

__global__ void __launch_bounds__(1024) lengths_kernel(PagedCheck c) {
  bool bad = false;
#pragma unroll 4
  for (int i = threadIdx.x; i < c.B; i += 1024) bad |= bad_length(c, i);
  const int st = __syncthreads_or(bad) ? TV_ERR_BAD_SEQLEN : 0;
  for (int i = threadIdx.x; i < c.B; i += 1024) c.err[i] = st;
}

__global__ void __launch_bounds__(256) paged_check_kernel(PagedCheck c) {
  plan_begun();
  int n;
  const int st = check_sequence(c, blockIdx.x, n);
  if (threadIdx.x == 0) c.err[blockIdx.x] = st;
}

}  // namespace

cudaError_t check_lengths(const PagedCheck& c, cudaStream_t s) {
  if (c.cu == nullptr || c.B <= kFewLengths) return cudaSuccess;
  lengths_kernel<<<1, 1024, 0, s>>>(c);
  return cudaGetLastError();
}

cudaError_t launch_paged_check(const PagedCheck& c, cudaStream_t s) {
  const cudaError_t e = check_lengths(c, s);
  if (e != cudaSuccess) return e;
  paged_check_kernel<<<c.B, 256, 0, s>>>(c);
  return cudaGetLastError();
}

}  // namespace tv
