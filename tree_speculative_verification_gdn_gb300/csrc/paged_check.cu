// Sequences of new tokens over a paged cache, checked before a call writes anything: the packed lengths, the room in
// the block table, and the blocks that the call writes to or that some new token sees.  A block a sequence; the packed
// lengths are read by every block, so that each can tell its own sequence's status alone.
#include "tv_common.cuh"
#include "tv_internal.h"

namespace tv {
namespace {

__global__ void __launch_bounds__(256) paged_check_kernel(PagedCheckArgs a) {
  const int b = blockIdx.x;
  for (int h = threadIdx.x; h < a.counters; h += blockDim.x) a.zeros[(long long)b * a.counters + h] = 0;
  bool bad = false;
  if (a.cu != nullptr)
    for (int i = threadIdx.x; i < a.B; i += blockDim.x) {
      const int lo = a.cu[i], hi = a.cu[i + 1];
      bad |= lo < 0 || hi < lo || hi > a.T || hi - lo > a.max_len;
    }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) a.err[b] = TV_ERR_BAD_SEQLEN;
    return;
  }
  const int n = a.cu != nullptr ? a.cu[b + 1] - a.cu[b] : 1;
  int st = 0;
  if (n > 0 && (a.live == nullptr || a.live[b] != 0)) {
    const int P = a.prefix_len != nullptr ? a.prefix_len[b] : 0;
    const long long room = a.table != nullptr ? (long long)a.max_blocks * 16 : 0x7fffffffLL;
    if (P < 0 || (long long)P + n > room) st = TV_ERR_CAPACITY;
    if (st == 0 && a.table != nullptr) {
      const int32_t* table = a.table + (long long)b * a.max_blocks;
      const int lo = a.window < 0 ? P : a.window > 0 ? max(0, P - a.window + 1) : 0;
      const int first = a.window < 0 ? 0 : (min(a.sinks, lo) + 15) / 16;  // pages of the first tokens
      bad = false;
      for (int i = threadIdx.x; i < first; i += blockDim.x) bad |= (unsigned)table[i] >= (unsigned)a.num_blocks;
      for (int i = lo / 16 + threadIdx.x; i <= (P + n - 1) / 16; i += blockDim.x)
        bad |= (unsigned)table[i] >= (unsigned)a.num_blocks;
      if (__syncthreads_or(bad)) st = TV_ERR_BAD_BLOCK;
    }
  }
  if (threadIdx.x == 0) a.err[b] = st;
}

}  // namespace

cudaError_t launch_paged_check(const PagedCheckArgs& a, cudaStream_t s) {
  paged_check_kernel<<<a.B, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace tv
