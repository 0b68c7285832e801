// What the kernels of the windowed attention share: which pages of a sequence some new token sees.
#pragma once

#include "tv_common.cuh"
#include "tv_internal.h"

namespace tv {

// New tokens of a sequence and the pages that they see between them, numbered without the hidden ones: first
// `front` pages of the first tokens, then those from logical page `from` on.
struct Seen {
  int n, P;     // new tokens (0: nothing to do), tokens before them
  int lo, s;    // first position in the first token's window; first tokens that stay visible before it
  int front, from, pages;
  __device__ int position(int page) const { return (page < front ? page : page - front + from) * 16; }
};

__device__ __forceinline__ Seen seen_by(const WinAttnArgs& a, int b) {
  Seen x;
  x.n = 0, x.pages = 0;
  if (a.err[b] != 0 || (a.live != nullptr && a.live[b] == 0)) return x;
  x.n = a.cu != nullptr ? a.cu[b + 1] - a.cu[b] : 1;
  if (x.n == 0) return x;
  x.P = a.prefix_len[b];
  x.lo = a.window > 0 ? max(0, x.P - a.window + 1) : 0;
  x.s = min(a.sinks, x.lo);
  x.front = (x.s + 15) / 16, x.from = x.lo / 16;
  if (x.from <= x.front) x.front = x.from = 0;  // nothing hidden between them
  x.pages = x.front + (x.P + x.n - 1) / 16 - x.from + 1;
  return x;
}

// Head dims 64, 128, 256; a.cu or one token a sequence.  Few rows: sequences of at most rows_limit(hd) query rows
// (new tokens x query heads of a KV head).
constexpr int rows_limit(int hd) { return 4096 / hd; }
size_t window_rows_workspace(int B, int Hkv, int rows, int hd);
cudaError_t launch_window_rows(const WinAttnArgs& a, void* workspace, cudaStream_t s);

}  // namespace tv
