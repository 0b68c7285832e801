// The elementwise rows around a mixer: the gated norm of its output per head, and the residual
// update with the norms before and after it.
//
// Both are bound by HBM: one pass, every row held in registers between its sum of squares and its
// scaling.  A row's columns are taken in vectors of eight that start on a 16-byte boundary of the
// first input, so a row of any length and offset reads and writes whole vectors except at its two
// ends; a tensor whose rows lie otherwise falls back to single elements where it must.
#include "tv_common.cuh"
#include "tv_internal.h"

namespace tv {
namespace {

template <typename T>
__device__ __forceinline__ bool vec_ok(const T* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// Columns e .. e + 7 of a row of n, zero outside it.  FULL: all inside, and aligned.
template <bool FULL, typename T>
__device__ __forceinline__ void load8(const T* row, int e, int n, float* x) {
  if (FULL || (e >= 0 && e + 8 <= n && vec_ok(row + e))) {
    load_vec_rw<8>(row + e, x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = e + i >= 0 && e + i < n ? to_f32(row[e + i]) : 0.f;
  }
}
template <bool FULL, typename T>
__device__ __forceinline__ void store8(T* row, int e, int n, const float* x) {
  if (FULL || (e >= 0 && e + 8 <= n && vec_ok(row + e))) {
    store_vec<8>(row + e, x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e + i >= 0 && e + i < n) row[e + i] = from_f32<T>(x[i]);
  }
}

// Elements from the 16-byte boundary at or before p to p.
template <typename T>
__device__ __forceinline__ int phase_of(const T* p) {
  return (int)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
}

// Sum over the G threads of a row: G <= 32 consecutive lanes, or (G = 0) the whole block.
template <int G>
__device__ __forceinline__ float row_sum(float x, float* s_part) {
  if constexpr (G > 0) {
    return group_sum<G>(x);
  } else {
    x = group_sum<32>(x);
    const int warps = blockDim.x / 32;
    __syncthreads();  // the previous sum's readers are done
    if (threadIdx.x % 32 == 0) s_part[threadIdx.x / 32] = x;
    __syncthreads();
    x = threadIdx.x % 32 < warps ? s_part[threadIdx.x % 32] : 0.f;
    return group_sum<32>(x);
  }
}

// g / (1 + exp(-g)), to the precision that the element type can show: bf16 keeps 2^-8 of a value, the
// hardware's 2^x and reciprocal are good to 2^-21 of it where the gate is not yet 0 or 1.  Reciprocals of more
// than 2^126 are 0 in both forms: silu of a gate below -87.3, at most 1e-36, is then 0.
__device__ __forceinline__ float2 silu2(float2 g, bf16) {
  constexpr float k = -1.4426950408889634f;  // -log2(e)
  const float2 x = __fmul2_rn(g, make_float2(k, k));
  float2 e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(x.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(x.y));
  e = __fadd2_rn(e, make_float2(1.f, 1.f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
  return __fmul2_rn(g, r);
}
__device__ __forceinline__ float2 silu2(float2 g, float) {
  return make_float2(__fdividef(g.x, 1.f + expf(-g.x)), __fdividef(g.y, 1.f + expf(-g.y)));
}

// id / H for ids below 2^31, by a multiplication: the quotient of every thread's row cost as much as
// half its arithmetic.
struct Divide {
  unsigned mul, shift;
};
Divide divide_by(int H) {
  unsigned s = 0;
  while ((1u << s) < (unsigned)H) ++s;  // 2^s >= H
  return {s == 0 ? 0u : (unsigned)((1ull << (31 + s)) / H + 1), s};
}
__device__ __forceinline__ int quotient(int id, Divide by) {
  return by.shift == 0 ? id : (int)(__umulhi((unsigned)id, by.mul) >> (by.shift - 1));
}

// G > 0: G lanes a row, one vector each, eight blocks on an SM to keep 64 KB of loads in flight
// (40001 x 32 rows of 128 bf16: 220 us without the bound on registers; two rows a thread 205 us).
// G = 0: a block a row, VPT vectors a thread.
template <typename T, int G, int VPT, bool FULL>
__global__ void __launch_bounds__(G == 0 ? 1024 : 256, G == 0 ? 1 : 8) gated_rmsnorm_kernel(GatedNormArgs a, Divide by) {
  __shared__ float s_part[32];
  const int per = G > 0 ? G : blockDim.x;
  const int id = G > 0 ? blockIdx.x * (256 / (G > 0 ? G : 1)) + threadIdx.x / per : blockIdx.x;
  const int l = G > 0 ? threadIdx.x % per : threadIdx.x;
  const bool in = id < a.rows * a.H;  // every lane stays for the sums
  const int r = in ? quotient(id, by) : 0, h = in ? id - r * a.H : 0;
  const int n = in ? a.d : 0;
  const T* x = static_cast<const T*>(a.x) + r * a.x_stride + (long long)h * a.d;
  const T* gate = a.gate != nullptr ? static_cast<const T*>(a.gate) + r * a.gate_stride + (long long)h * a.d : nullptr;
  const T* w = static_cast<const T*>(a.weight);
  T* out = static_cast<T*>(a.out) + r * a.out_stride + (long long)h * a.d;
  const int phase = FULL ? 0 : phase_of(x);
  // Columns in pairs: one by one the kernel issued an instruction four clocks in five (170 us, now 166).
  float2 v[VPT][4], g[VPT][4], sum2 = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int e = (l + j * per) * 8 - phase;
    if (e >= n) continue;
    load8<FULL>(x, e, n, &v[j][0].x);
    if (gate != nullptr) load8<FULL>(gate, e, n, &g[j][0].x);
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    if ((l + j * per) * 8 - phase >= n) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      g[j][i] = gate != nullptr ? silu2(g[j][i], T()) : make_float2(1.f, 1.f);
      if (a.gate_first) v[j][i] = __fmul2_rn(v[j][i], g[j][i]);
      sum2 = __ffma2_rn(v[j][i], v[j][i], sum2);
    }
  }
  const float root = rsqrtf(row_sum<G>(sum2.x + sum2.y, s_part) / a.d + a.eps);
  const float2 inv = make_float2(root, root), offset = make_float2(a.weight_offset, a.weight_offset);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int e = (l + j * per) * 8 - phase;
    if (e >= n) continue;
    float2 c[4];
    if (w != nullptr) load8<FULL>(w, e, n, &c[0].x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 y = __fmul2_rn(v[j][i], inv);
      if (w != nullptr) y = __fmul2_rn(y, __fadd2_rn(offset, c[i]));
      v[j][i] = a.gate_first ? y : __fmul2_rn(y, g[j][i]);
    }
    store8<FULL>(out, e, n, &v[j][0].x);
  }
}

// A block a row, a vector a thread up to 8192 columns (wider rows take five, and spill): y, gate and
// residual are asked for at once, then two sums with a block's barriers each.  Bound by HBM: 30011 rows of
// 5120 with an fp32 residual, both norms and a gate 349 us = 6.2 TB/s, 0.91 of a plain copy's rate; two
// vectors a thread 399 us.
template <typename T, typename TR, int VPT, bool FULL>
__global__ void __launch_bounds__(1024) residual_rmsnorm_kernel(ResidualNormArgs a) {
  __shared__ float s_part[32];
  const int n = a.D, per = blockDim.x, l = threadIdx.x;
  const long long r = blockIdx.x;
  const T* y = static_cast<const T*>(a.y) + r * a.y_stride;
  const TR* res = static_cast<const TR*>(a.residual) + r * a.residual_stride;
  const T* gate = a.gate != nullptr ? static_cast<const T*>(a.gate) + r * a.gate_stride : nullptr;
  const T* pw = static_cast<const T*>(a.post_weight);
  const T* w = static_cast<const T*>(a.weight);
  TR* ro = static_cast<TR*>(a.residual_out) + r * a.residual_out_stride;
  T* out = a.out != nullptr ? static_cast<T*>(a.out) + r * a.out_stride : nullptr;
  const int phase = FULL ? 0 : phase_of(y);
  float t[VPT][8], x[VPT][8], g[VPT][8];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int e = (l + j * per) * 8 - phase;
    if (e >= n) continue;
    load8<FULL>(y, e, n, t[j]);
    load8<FULL>(res, e, n, x[j]);
    if (gate != nullptr) load8<FULL>(gate, e, n, g[j]);
  }
  float inv = 1.f;
  if (pw != nullptr) {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if ((l + j * per) * 8 - phase >= n) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(t[j][i], t[j][i], sum);
    }
    inv = rsqrtf(row_sum<0>(sum, s_part) / n + a.eps);
  }
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int e = (l + j * per) * 8 - phase;
    if (e >= n) continue;
    float c[8];
    if (pw != nullptr) load8<FULL>(pw, e, n, c);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float u = t[j][i];
      if (pw != nullptr) u *= inv * (a.weight_offset + c[i]);
      if (gate != nullptr) u *= g[j][i];
      x[j][i] = fmaf(a.scale, u, x[j][i]);
      if (FULL || (e + i >= 0 && e + i < n)) sum = fmaf(x[j][i], x[j][i], sum);
    }
    store8<FULL>(ro, e, n, x[j]);
  }
  if (out == nullptr) return;
  inv = rsqrtf(row_sum<0>(sum, s_part) / n + a.eps);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int e = (l + j * per) * 8 - phase;
    if (e >= n) continue;
    float c[8];
    if (w != nullptr) load8<FULL>(w, e, n, c);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[j][i] *= inv;
      if (w != nullptr) x[j][i] *= a.weight_offset + c[i];
    }
    store8<FULL>(out, e, n, x[j]);
  }
}

// Every row of the tensor starts on a 16-byte boundary.
bool rows16(const void* p, long long stride, int dtype) {
  return p == nullptr ||
         ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && stride * (dtype == TV_F32 ? 4 : 2) % 16 == 0);
}

template <typename T, int G, int VPT>
cudaError_t gated_go(const GatedNormArgs& a, bool full, int block, cudaStream_t s) {
  constexpr int per = G > 0 ? 256 / (G > 0 ? G : 1) : 1;
  const unsigned grid = (unsigned)(((long long)a.rows * a.H + per - 1) / per);
  const Divide by = divide_by(a.H);
  if (full) gated_rmsnorm_kernel<T, G, VPT, true><<<grid, block, 0, s>>>(a, by);
  else gated_rmsnorm_kernel<T, G, VPT, false><<<grid, block, 0, s>>>(a, by);
  return cudaGetLastError();
}

template <typename T>
cudaError_t gated(const GatedNormArgs& a, cudaStream_t s) {
  const bool full = a.d % 8 == 0 && rows16(a.x, a.x_stride, a.io) && rows16(a.gate, a.gate_stride, a.io) &&
                    rows16(a.weight, 0, a.io) && rows16(a.out, a.out_stride, a.io);
  const int vecs = full ? a.d / 8 : (a.d + 14) / 8;  // a row at an offset can touch one vector more
  if (vecs <= 8) return gated_go<T, 8, 1>(a, full, 256, s);
  if (vecs <= 16) return gated_go<T, 16, 1>(a, full, 256, s);
  if (vecs <= 32) return gated_go<T, 32, 1>(a, full, 256, s);
  const int vpt = (vecs + 1023) / 1024;
  const int block = ((vecs + vpt - 1) / vpt + 31) / 32 * 32;
  if (vpt == 1) return gated_go<T, 0, 1>(a, full, block, s);
  return gated_go<T, 0, 5>(a, full, block, s);
}

template <typename T, typename TR, int VPT>
cudaError_t residual_go(const ResidualNormArgs& a, bool full, int block, cudaStream_t s) {
  if (full) residual_rmsnorm_kernel<T, TR, VPT, true><<<a.rows, block, 0, s>>>(a);
  else residual_rmsnorm_kernel<T, TR, VPT, false><<<a.rows, block, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T, typename TR>
cudaError_t residual(const ResidualNormArgs& a, cudaStream_t s) {
  const bool full = a.D % 8 == 0 && rows16(a.y, a.y_stride, a.io) && rows16(a.gate, a.gate_stride, a.io) &&
                    rows16(a.residual, a.residual_stride, a.res) &&
                    rows16(a.residual_out, a.residual_out_stride, a.res) && rows16(a.out, a.out_stride, a.io) &&
                    rows16(a.weight, 0, a.io) && rows16(a.post_weight, 0, a.io);
  const int vecs = full ? a.D / 8 : (a.D + 14) / 8;
  const int vpt = (vecs + 1023) / 1024;
  const int block = ((vecs + vpt - 1) / vpt + 31) / 32 * 32;
  if (vpt == 1) return residual_go<T, TR, 1>(a, full, block, s);
  return residual_go<T, TR, 5>(a, full, block, s);
}

}  // namespace

cudaError_t launch_gated_rmsnorm(const GatedNormArgs& a, cudaStream_t s) {
  return a.io == TV_F32 ? gated<float>(a, s) : gated<bf16>(a, s);
}

cudaError_t launch_residual_rmsnorm(const ResidualNormArgs& a, cudaStream_t s) {
  if (a.io == TV_F32) return residual<float, float>(a, s);
  return a.res == TV_BF16 ? residual<bf16, bf16>(a, s) : residual<bf16, float>(a, s);
}

}  // namespace tv
