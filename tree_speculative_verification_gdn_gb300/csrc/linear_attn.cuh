// How the prompt kernels of linear attention find their work: packed prompts, cut into segments
// where they are long.
#pragma once

#include "tv_common.cuh"
#include "tv_internal.h"

namespace tv {

// Every entry of cu_seqlens ascends inside [0, T] and no prompt is longer than max_len; the same
// answer in every thread.  Only then do the segments below stay inside the workspace:
// sum max(1, ceil(len / seg_len)) <= B + T / seg_len.  Contains __syncthreads().
__device__ __forceinline__ bool check_seqlens(const LinAttnArgs& a) {
  bool bad = false;
  for (int i = threadIdx.x; i < a.B; i += blockDim.x) {
    const int lo = __ldg(a.cu + i), hi = __ldg(a.cu + i + 1);
    bad |= lo < 0 || hi < lo || hi > a.T || hi - lo > a.max_len;
  }
  return !__syncthreads_or(bad);
}

struct Segment {
  int b;        // prompt; -1: no such segment (empty, the other fields set)
  int h;        // value head
  int index;    // segment of the prompt
  int count;    // segments of the prompt
  int t0, t1;   // its tokens
};

__device__ __forceinline__ int segments_of(int len, int seg_len) {
  return seg_len > 0 && len > seg_len ? (len + seg_len - 1) / seg_len : 1;
}

// Unit u is head u % H of segment u / H, segments counted over all prompts.  Executed by a whole warp,
// the same answer in every lane; cu_seqlens has passed check_seqlens.
static __device__ __noinline__ Segment find_segment(const LinAttnArgs& a, int u) {
  const int g = u / a.H;
  Segment s{-1, u - g * a.H, 0, 1, 0, 0};
  if (a.seg_len == 0) {
    if (g < a.B) {
      s.b = g;
      s.index = 0;
      s.count = 1;
      s.t0 = __ldg(a.cu + g);
      s.t1 = __ldg(a.cu + g + 1);
    }
    return s;
  }
  const int lane = threadIdx.x & 31;
  int base = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    const int lo = b < a.B ? __ldg(a.cu + b) : 0, hi = b < a.B ? __ldg(a.cu + b + 1) : 0;
    const int n = b < a.B ? segments_of(hi - lo, a.seg_len) : 0;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    const unsigned past = __ballot_sync(0xffffffffu, base + sum > g);
    if (past) {
      const int at = __ffs(past) - 1;
      s.b = b0 + at;
      s.count = __shfl_sync(0xffffffffu, n, at);
      s.index = g - base - (__shfl_sync(0xffffffffu, sum, at) - s.count);
      const int t = __shfl_sync(0xffffffffu, lo, at), end = __shfl_sync(0xffffffffu, hi, at);
      s.t0 = t + s.index * a.seg_len;
      s.t1 = s.index + 1 < s.count ? s.t0 + a.seg_len : end;
      return s;
    }
    base += __shfl_sync(0xffffffffu, sum, 31);
  }
  return s;
}

// First segment number of prompt b (warp-wide, as above).
__device__ __forceinline__ int first_segment(const LinAttnArgs& a, int b) {
  const int lane = threadIdx.x & 31;
  int sum = 0;
  for (int i = lane; i < b; i += 32) sum += segments_of(__ldg(a.cu + i + 1) - __ldg(a.cu + i), a.seg_len);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

}  // namespace tv
