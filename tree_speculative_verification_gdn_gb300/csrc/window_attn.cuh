// What the kernels of the windowed attention share: which keys some new token sees, and how the work is dealt out.
#pragma once

#include "tv_common.cuh"
#include "tv_internal.h"
#include "tv_launch.cuh"

namespace tv {

// A run of new tokens of one sequence, and the pages that they see between them, numbered without the hidden ones:
// first `front` pages of the first tokens, then those from logical page `from` on.
struct Seen {
  int n, P;     // tokens (0: nothing to do), tokens before them
  int lo, s;    // first position in the first token's window; first tokens that stay visible before it
  int front, from, pages;
  __device__ int position(int page) const { return (page < front ? page : page - front + from) * 16; }
};

__device__ __forceinline__ Seen seen_by(const WinAttnArgs& a, int P, int n) {
  Seen x;
  x.n = n, x.P = P;
  x.lo = a.window > 0 ? max(0, P - a.window + 1) : 0;
  x.s = min(a.sinks, x.lo);
  x.front = (x.s + 15) / 16, x.from = x.lo / 16;
  if (x.from <= x.front) x.front = x.from = 0;  // nothing hidden between them
  x.pages = x.front + (P + n - 1) / 16 - x.from + 1;
  return x;
}

constexpr int kSms = 152;

// a / b of numbers that hardly ever need 64 bits
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return (((unsigned long long)a | (unsigned long long)b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// The costs of all sequences, Hkv times each, lie one behind the other; CTA i of the grid takes the i-th of equal runs of
// at least `least`.
struct Run {
  long long per, x0, x1;  // a run's length; this CTA's
  int b;                  // the sequence that it starts in, and the cost before that
  long long base;
  int start, n, P;        // first token, tokens, and tokens before them, of that sequence
};
// The whole block; false in every thread where the run is empty.  THREADS = blockDim.x.  What up to THREADS sequences need is
// asked for at once: a short call is a chain of such latencies.
template <int THREADS>
__device__ __forceinline__ bool find_run(const WinAttnArgs& a, const long long* cost, int least, Run& r) {
  constexpr int W = THREADS / 32;
  __shared__ long long part[2][W];
  __shared__ Run found;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  // sum over the block; upto: over the threads before this one and it
  int turn = 0;
  auto scan = [&](long long x, long long& upto) -> long long {
    upto = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) part[turn][warp] = upto;
    __syncthreads();
    long long all = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < warp) upto += part[turn][w];
      all += part[turn][w];
    }
    turn ^= 1;
    return all;
  };
  auto tokens_of = [&](int b, int& start, int& n, int& P) {
    start = a.cu != nullptr ? a.cu[b] : b;
    n = (a.cu != nullptr ? a.cu[b + 1] : b + 1) - start;
    P = a.prefix_len[b];
  };
  const bool few = a.B <= THREADS;
  long long mine = 0, upto;
  int start = 0, n = 0, P = 0;
  for (int b = tid; b < a.B; b += THREADS) {
    mine += cost[b] * a.Hkv;
    if (few) tokens_of(b, start, n, P);
  }
  const long long total = scan(mine, upto);
  r.per = quotient(total + gridDim.x - 1, gridDim.x);
  if (r.per < least) r.per = least;
  r.x0 = blockIdx.x * r.per, r.x1 = min(total, r.x0 + r.per);
  if (r.x0 >= r.x1) return false;
  r.base = 0;
  for (int b0 = 0;; b0 += THREADS) {
    long long own = mine, here = total;
    if (!few) {
      own = b0 + tid < a.B ? cost[b0 + tid] * a.Hkv : 0;
      here = scan(own, upto);
    }
    if (r.base + here > r.x0) {
      if (r.base + upto - own <= r.x0 && r.base + upto > r.x0) {
        if (!few) tokens_of(b0 + tid, start, n, P);
        found.b = b0 + tid, found.base = r.base + upto - own;
        found.start = start, found.n = n, found.P = P;
      }
      break;
    }
    r.base += here;
  }
  __syncthreads();
  r.b = found.b, r.base = found.base;
  r.start = found.start, r.n = found.n, r.P = found.P;
  return true;
}

// Head dims 64, 128, 256; a.cu or one token a sequence.  cost [B]: of a sequence for one KV head.
// Few rows: at most 16 query rows (new tokens x query heads of a KV head) in a sequence; cost: pages.  With 32 rows of
// head dim 128 (32 chains of eight tokens behind 8192) this kernel took 117 us, that for any number 91 us.
// arrived [B * Hkv], zero; slots: bytes as window_rows_slots.
constexpr int kFewRows = 16;
size_t window_rows_slots(int hd);
cudaError_t launch_window_rows(const WinAttnArgs& a, const long long* cost, int* arrived, float* slots, cudaStream_t s);

// Any number of rows: units of `tokens` tokens; cost: per unit its key tiles and kUnitCost more.  One prompt of 4096 tokens, 32
// heads on 8 of 128: 153 us with 2 for that, 134 with 4, 135 with 7.
struct TileShape {
  int tokens;  // of a unit
  int keys;    // of a tile
};
constexpr int kUnitCost = 4;
TileShape window_tile_shape(int Hq, int Hkv, int hd);
// arrived [kSms * 8], zero; slots: bytes as window_tiles_slots.
size_t window_tiles_slots(int hd);
cudaError_t launch_window_tiles(const WinAttnArgs& a, const long long* cost, int* arrived, float* slots, cudaStream_t s);

}  // namespace tv
