// Sequences of new tokens over a paged cache, checked before a call writes anything: the packed lengths, the room in
// the block table, and the blocks that the call writes to or that some new token sees.  A block a sequence.  Up to kFewLengths
// sequences every block reads all the packed lengths, so that each can tell its own sequence's status alone; past that
// one block reads them first, or the work would grow by the square of their number.
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
  int32_t* err;               // [B]; more than kFewLengths sequences: holds what check_lengths found
};

// 512 tokens rotated into the cache, 1024 sequences: 14.0 us with every block reading, 14.8 with one first; 2048 sequences 17.2
// and 13.8; 262144 sequences 42.5 ms and 0.46.
constexpr int kFewLengths = 1024;

__device__ __forceinline__ bool bad_length(const PagedCheck& a, int i) {
  const int lo = a.cu[i], hi = a.cu[i + 1];
  return lo < 0 || hi < lo || hi > a.T || hi - lo > a.max_len;
}

// The status of sequence b, the same in every thread of the block; n: its new tokens, 0 where there is nothing to do.
__device__ __forceinline__ int check_sequence(const PagedCheck& a, int b, int& n) {
  n = 0;
  bool bad = false;
  if (a.cu != nullptr) {
    if (a.B > kFewLengths) bad = threadIdx.x == 0 && a.err[b] == TV_ERR_BAD_SEQLEN;
    else for (int i = threadIdx.x; i < a.B; i += blockDim.x) bad |= bad_length(a, i);
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

// Before any kernel that calls check_sequence.
cudaError_t check_lengths(const PagedCheck& c, cudaStream_t s);
// err[b] of every sequence, by the check alone.
cudaError_t launch_paged_check(const PagedCheck& c, cudaStream_t s);

}  // namespace tv
