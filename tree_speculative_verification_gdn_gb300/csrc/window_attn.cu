// GQA attention of new tokens over the paged cache, within a window and to a few first tokens.
//
// o = sum_j softmax_j(scale q . k_j) v_j over the keys j <= p of a query at position p with p - j < window, or
// j < sinks.  A warp takes one query head of one token and walks its keys with a running maximum and sum.
#include "window_attn.cuh"

namespace tv {
namespace {

template <int HD>
__global__ void __launch_bounds__(256) window_attn_kernel(WinAttnArgs a) {
  constexpr int E = HD / 32;
  const int lane = threadIdx.x % 32;
  const long long id = (long long)blockIdx.x * 8 + threadIdx.x / 32;
  const int t = (int)(id / a.Hq), h = (int)(id % a.Hq);
  if (t >= a.T) return;
  int b = t, p = 0;
  if (a.cu != nullptr) {
    if (a.err[0] == TV_ERR_BAD_SEQLEN) return;
    int n = 0;
    for (int i = lane; i <= a.B; i += 32) n += a.cu[i] <= t;
    b = __reduce_add_sync(0xffffffffu, n) - 1;
    if (b < 0 || b >= a.B) return;
    p = t - a.cu[b];
  }
  if (a.err[b] != 0 || (a.live != nullptr && a.live[b] == 0)) return;
  p += a.prefix_len[b];
  const int32_t* table = a.block_table + (long long)b * a.max_blocks;
  const int kvh = h / (a.Hq / a.Hkv);
  float q[E], o[E], m = -INFINITY, l = 0.f;
  const bf16* qp = static_cast<const bf16*>(a.q) + t * a.q_stride + h * HD + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) q[e] = to_f32(qp[e]) * (a.sm_scale * 1.4426950408889634f), o[e] = 0.f;
  const int lo = a.window > 0 ? max(0, p - a.window + 1) : 0;
  for (int j = lo == 0 || a.sinks == 0 ? lo : 0; j <= p; ++j) {
    if (j < lo && j >= a.sinks) j = lo;
    const long long row = ((long long)table[j / 16] * a.Hkv + kvh) * 16 + j % 16;
    const bf16* kp = static_cast<const bf16*>(a.k_cache) + row * HD + lane * E;
    const bf16* vp = static_cast<const bf16*>(a.v_cache) + row * HD + lane * E;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], to_f32(kp[e]), s);
    s = group_sum<32>(s);
    const float mn = fmaxf(m, s), f = exp2f(m - mn), w = exp2f(s - mn);
    l = l * f + w, m = mn;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], f, w * to_f32(vp[e]));
  }
  bf16* op = static_cast<bf16*>(a.out) + t * a.out_stride + h * HD + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) op[e] = from_f32<bf16>(o[e] / l);
}

}  // namespace

size_t window_attn_workspace_size(int B, int T, int max_len, int Hq, int Hkv, int hd, int max_blocks, int window,
                                  int sinks) {
  const long long rows = (long long)max_len * (Hq / Hkv);
  if (T == 0) return 0;
  return rows <= rows_limit(hd) ? window_rows_workspace(B, Hkv, (int)rows, hd) : 0;
}

cudaError_t launch_window_attn(const WinAttnArgs& a, void* workspace, cudaStream_t s) {
  const bool few = a.T > 0 && (long long)a.max_len * (a.Hq / a.Hkv) <= rows_limit(a.hd);
  const PagedCheckArgs c{a.cu, a.prefix_len, a.live, a.block_table, a.B, a.T, a.max_len, a.max_blocks, a.num_blocks,
                         a.window, a.sinks, a.err, static_cast<int32_t*>(workspace), few ? a.Hkv : 0};
  const cudaError_t e = launch_paged_check(c, s);
  if (e != cudaSuccess || a.T == 0) return e;
  if (few) return launch_window_rows(a, workspace, s);
  const unsigned grid = (unsigned)(((long long)a.T * a.Hq + 7) / 8);
  if (a.hd == 64) window_attn_kernel<64><<<grid, 256, 0, s>>>(a);
  else if (a.hd == 128) window_attn_kernel<128><<<grid, 256, 0, s>>>(a);
  else window_attn_kernel<256><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace tv
