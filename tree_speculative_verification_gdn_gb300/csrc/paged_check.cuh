// Sequences of new tokens over a paged cache, checked before a call writes anything: the packed lengths, the room in
// the block table, and the blocks that the call writes to or that some new token sees.  A block a sequence; the packed
// lengths are read by every block, so that each can tell its own sequence's status alone.
#pragma once

#include "tv_common.cuh"

namespace tv {

struct PagedCheck {
  const int32_t* cu;          // [B + 1], or nullptr: one token a sequence
  const int32_t* prefix_len;  // nullptr: zero
  const int32_t* live;        // nullptr: all
  const int32_t* table;       // nullptr: no cache
  int B, T, max_len, max_blocks, num_blocks;
  int window;                 // < 0: the blocks of the new tokens, else those that they see
  int sinks;
};

// The status of sequence b, the same in every thread of the block; n: its new tokens, 0 where there is nothing to do.
__device__ __forceinline__ int check_sequence(const PagedCheck& a, int b, int& n) {
  n = 0;
  bool bad = false;
  if (a.cu != nullptr)
    for (int i = threadIdx.x; i < a.B; i += blockDim.x) {
      const int lo = a.cu[i], hi = a.cu[i + 1];
      bad |= lo < 0 || hi < lo || hi > a.T || hi - lo > a.max_len;
    }
  if (__syncthreads_or(bad)) return TV_ERR_BAD_SEQLEN;
  const int tokens = a.cu != nullptr ? a.cu[b + 1] - a.cu[b] : 1;
  if (tokens == 0 || (a.live != nullptr && a.live[b] == 0)) return 0;
  const int P = a.prefix_len != nullptr ? a.prefix_len[b] : 0;
  const long long room = a.table != nullptr ? (long long)a.max_blocks * 16 : 0x7fffffffLL;
  if (P < 0 || (long long)P + tokens > room) return TV_ERR_CAPACITY;
  if (a.table != nullptr) {
    const int32_t* table = a.table + (long long)b * a.max_blocks;
    const int lo = a.window < 0 ? P : a.window > 0 ? max(0, P - a.window + 1) : 0;
    const int first = a.window < 0 ? 0 : (min(a.sinks, lo) + 15) / 16;  // pages of the first tokens
    bad = false;
    for (int i = threadIdx.x; i < first; i += blockDim.x) bad |= (unsigned)table[i] >= (unsigned)a.num_blocks;
    for (int i = lo / 16 + threadIdx.x; i <= (P + tokens - 1) / 16; i += blockDim.x)
      bad |= (unsigned)table[i] >= (unsigned)a.num_blocks;
    if (__syncthreads_or(bad)) return TV_ERR_BAD_BLOCK;
  }
  n = tokens;
  return 0;
}

// err[b] of every sequence, by the check alone.
cudaError_t launch_paged_check(const PagedCheck& c, int32_t* err, cudaStream_t s);

}  // namespace tv
