// GQA attention of new tokens over the paged cache, within a window and to a few first tokens.
//
// o = sum_j softmax_j(scale q . k_j) v_j over the keys j <= p of a query at position p with p - j < window, or
// j < sinks.  Two launches: a plan, which checks every sequence before anything is written, counts its work and clears
// the counters of shared outputs; then one of two kernels that read the visible pages alone, by the number of query
// rows that a key is read for.
#include "paged_check.cuh"
#include "window_attn.cuh"

namespace tv {
namespace {

// A block a sequence.  shape.tokens = 0: its cost is its pages.
__global__ void __launch_bounds__(256) window_plan_kernel(WinAttnArgs a, PagedCheck c, TileShape shape,
                                                          long long* __restrict__ cost, int* __restrict__ zeros, int count) {
  plan_begun();
  const int b = blockIdx.x;
  for (long long i = (long long)b * 256 + threadIdx.x; i < count; i += (long long)a.B * 256) zeros[i] = 0;
  int n;
  const int st = check_sequence(c, b, n);
  __shared__ long long part[8];
  long long sum = 0;
  if (n > 0 && shape.tokens == 0) {
    if (threadIdx.x == 0) sum = seen_by(a, a.prefix_len[b], n).pages;
  } else if (n > 0) {
    for (long long t = (long long)threadIdx.x * shape.tokens; t < n; t += 256LL * shape.tokens) {
      const int pages = seen_by(a, a.prefix_len[b] + (int)t, min(shape.tokens, n - (int)t)).pages;
      sum += (pages * 16 + shape.keys - 1) / shape.keys + kUnitCost;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0;
    for (int w = 0; w < 8; ++w) sum += part[w];
    cost[b] = sum;
    a.err[b] = st;
  }
}

size_t align16(size_t x) { return (x + 15) & ~(size_t)15; }
bool few_rows(int max_len, int group) { return (long long)max_len * group <= kFewRows; }
// workspace: costs, counters, slots of shared outputs
int counters(int B, int Hkv, bool few) { return few ? B * Hkv : kSms * 8; }

}  // namespace

size_t window_attn_workspace_size(int B, int T, int max_len, int Hq, int Hkv, int hd, int max_blocks, int window,
                                  int sinks) {
  if (T == 0) return 0;
  const bool few = few_rows(max_len, Hq / Hkv);
  return align16((size_t)B * 8) + align16((size_t)counters(B, Hkv, few) * 4) +
         (few ? window_rows_slots(hd) : window_tiles_slots(hd));
}

cudaError_t launch_window_attn(const WinAttnArgs& a, void* workspace, cudaStream_t s) {
  const bool few = few_rows(a.max_len, a.Hq / a.Hkv);
  const PagedCheck c{a.cu, a.prefix_len, a.live, a.block_table, a.B, a.T, a.max_len, a.max_blocks, a.num_blocks,
                     a.window, a.sinks, a.err};
  if (a.T == 0) return launch_paged_check(c, s);  // no workspace
  long long* cost = static_cast<long long*>(workspace);
  int* zeros = reinterpret_cast<int*>(static_cast<char*>(workspace) + align16((size_t)a.B * 8));
  const int count = counters(a.B, a.Hkv, few);
  const TileShape shape = few ? TileShape{0, 0} : window_tile_shape(a.Hq, a.Hkv, a.hd);
  cudaError_t e = check_lengths(c, s);
  if (e != cudaSuccess) return e;
  window_plan_kernel<<<a.B, 256, 0, s>>>(a, c, shape, cost, zeros, count);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  float* slots = reinterpret_cast<float*>(reinterpret_cast<char*>(zeros) + align16((size_t)count * 4));
  return few ? launch_window_rows(a, cost, zeros, slots, s) : launch_window_tiles(a, cost, zeros, slots, s);
}

}  // namespace tv
