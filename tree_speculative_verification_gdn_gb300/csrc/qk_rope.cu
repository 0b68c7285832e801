// Norms of queries and keys per head, their rotation by position, and the new keys and values into the paged cache.
//
// y = x / sqrt(mean(x^2) + eps) * (offset + w) over a head's hd columns, then pairs (y_c, y_{c + r/2}), c < r/2, turned
// by position * theta^(-2c/r).  HD / 16 lanes take a head, each two vectors of eight columns that lie r/2 apart, so
// that a pair meets in one thread; columns past r come as two neighbouring vectors.
//
// Angles: theta^(-2c/r) / 2 pi is a fraction of a turn for each position.  In 64-bit fixed point position times that
// fraction drops whole turns by its overflow, exactly, however far the position; the nearest quarter turn comes off as
// two bits and what is left, an eighth of a turn at most, goes to sincospi with its 24 bits whole.  They are made once
// a token, by the threads of its heads, a token ahead of their use.
//
// Bound by HBM: q, k and v are read once and written once.  A block walks a run of tokens with the next one's vectors
// already asked for; its place among the sequences is searched once, then counted on.
#include <math.h>

#include "paged_check.cuh"
#include "tv_common.cuh"
#include "tv_internal.h"

namespace tv {
namespace {

struct Turns {
  unsigned long long f[128];  // turns a position, in 2^-64
};

template <typename T>
struct Vectors;  // two vectors of eight columns as they lie in memory
template <>
struct Vectors<bf16> {
  uint4 a, b;
  __device__ void load(const bf16* p, int second) {
    a = *reinterpret_cast<const uint4*>(p);
    b = *reinterpret_cast<const uint4*>(p + second);
  }
  __device__ void get(float* x) const { unpack8(a, x), unpack8(b, x + 8); }
};
template <>
struct Vectors<float> {
  float4 v[4];
  __device__ void load(const float* p, int second) {
    v[0] = reinterpret_cast<const float4*>(p)[0], v[1] = reinterpret_cast<const float4*>(p)[1];
    v[2] = reinterpret_cast<const float4*>(p + second)[0], v[3] = reinterpret_cast<const float4*>(p + second)[1];
  }
  __device__ void get(float* x) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[4 * i] = v[i].x, x[4 * i + 1] = v[i].y, x[4 * i + 2] = v[i].z, x[4 * i + 3] = v[i].w;
  }
};

// The sequence of a token, its position and the row of its keys in the cache.
struct Place {
  int b, end;        // sequence (-1: before the first, B: past the last), and the token past its last
  int position;      // valid if go
  long long row;     // block * Hkv * 16 + position % 16, in rows of hd
  bool go;
};

// tpb tokens side by side, ipb heads (queries, keys, and with a cache values) of each; per_block tokens a block.
template <typename T, int HD>
__global__ void __launch_bounds__(512)
    qk_rope_kernel(const __grid_constant__ QkRopeArgs a, const __grid_constant__ Turns turns, int ipb, int tpb,
                   int per_block) {
  constexpr int L = HD / 16;
  extern __shared__ float2 s_cs[];  // (cos, sin) [2][tpb][rotary / 2]
  const int half = a.rotary / 2;
  const bool cache = a.k_cache != nullptr;
  const int items = a.Hq + (cache ? 2 : 1) * a.Hkv;
  const int u = threadIdx.x / L, l = threadIdx.x % L;
  const int tl = u / ipb, item = u % ipb + blockIdx.y * ipb;
  const bool in = tl < tpb;
  const bool mine = in && item < items;
  // 0: a query head, 1: a key head, 2: a value head
  const int kind = item < a.Hq ? 0 : item < a.Hq + a.Hkv ? 1 : 2;
  const int head = kind == 0 ? item : kind == 1 ? item - a.Hq : item - a.Hq - a.Hkv;
  const long long t0 = (long long)blockIdx.x * per_block;
  const int t1 = (int)min((long long)a.T, t0 + per_block);
  if (t0 >= t1) return;

  // columns first .. first + 7 and second further on
  const bool turns_here = l < a.rotary / 16;
  const int first = turns_here ? 8 * l : a.rotary + 16 * (l - a.rotary / 16);
  const int second = turns_here ? half : 8;
  const T* x_in = static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v);
  const long long x_stride = kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride;
  const T* weight = static_cast<const T*>(kind == 0 ? a.q_weight : a.k_weight);

  Place at;
  at.b = -1, at.end = 0, at.go = false;
  if (a.cu != nullptr) {
    if (a.err[0] == TV_ERR_BAD_SEQLEN) return;
    // the sequences that end at or before the block's first token lie behind it
    int n = 0;
    for (int i = threadIdx.x % 32; i <= a.B; i += 32) n += a.cu[i] <= t0;
    n = __reduce_add_sync(0xffffffffu, n);
    at.b = n - 1;
    at.end = n <= a.B ? a.cu[n] : 0x7fffffff;
  }
  auto find = [&](int t) {  // tokens come in ascending order
    at.go = false;
    if (t >= t1 || !in) return;
    if (a.cu != nullptr) {
      while (at.b < a.B && t >= at.end) {
        ++at.b;
        at.end = at.b < a.B ? a.cu[at.b + 1] : 0x7fffffff;
      }
      if (at.b < 0 || at.b >= a.B || a.err[at.b] != 0 || (a.live != nullptr && a.live[at.b] == 0)) return;
      at.position = (a.prefix_len != nullptr ? a.prefix_len[at.b] : 0) + t - a.cu[at.b];
    } else {
      at.b = t;
      int st = 0;
      const bool live = a.live == nullptr || a.live[t] != 0;
      at.position = a.prefix_len != nullptr ? a.prefix_len[t] : 0;
      if (live && (at.position < 0 || at.position >= (cache ? a.max_blocks * 16 : 0x7fffffff))) st = TV_ERR_CAPACITY;
      if (live && st == 0 && cache &&
          (unsigned)a.block_table[(long long)t * a.max_blocks + at.position / 16] >= (unsigned)a.num_blocks)
        st = TV_ERR_BAD_BLOCK;
      if (item == 0 && l == 0) a.err[t] = st;
      if (!live || st != 0) return;
    }
    if (cache)
      at.row = (long long)a.block_table[(long long)at.b * a.max_blocks + at.position / 16] * a.Hkv * 16 + at.position % 16;
    at.go = true;
  };
  auto angles = [&](int buf) {
    if (!at.go) return;
    float2* cs = s_cs + (buf * tpb + tl) * half;
    for (int c = (u - tl * ipb) * L + l; c < half; c += ipb * L) {
      const unsigned long long turn = (unsigned long long)(unsigned)at.position * turns.f[c];
      const unsigned long long quarter = (turn + (1ull << 61)) >> 62;
      const int rest = (int)((long long)(turn - (quarter << 62)) >> 30);  // in 2^-34 of a turn
      float sn, cn;
      sincospif((float)rest * 0x1p-33f, &sn, &cn);
      const float2 even = make_float2(cn, sn), odd = make_float2(-sn, cn);
      float2 v = quarter & 1 ? odd : even;
      if (quarter & 2) v.x = -v.x, v.y = -v.y;
      cs[c] = v;
    }
  };

  Vectors<T> now, next;
  int t = (int)t0 + tl;
  find(t);
  if (at.go && mine) now.load(x_in + t * x_stride + head * HD + first, second);
  angles(0);
  __syncthreads();
  int buf = 0;
  for (int base = (int)t0; base < t1; base += tpb, buf ^= 1) {
    const bool go = at.go && mine;
    const long long row = at.row;
    find(t + tpb);
    if (at.go && mine) next.load(x_in + (t + tpb) * x_stride + head * HD + first, second);
    angles(buf ^ 1);
    float x[16];
    float sum = 0.f;
    if (go) {
      now.get(x);
#pragma unroll
      for (int i = 0; i < 16; ++i) sum = fmaf(x[i], x[i], sum);
    }
    sum = group_sum<L>(sum);
    if (go) {
      if (kind != 2 && a.norm) {
        const float inv = rsqrtf(sum / HD + a.eps);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] *= inv;
        if (weight != nullptr) {
          float w[16];
          load_vec<8>(weight + first, w);
          load_vec<8>(weight + first + second, w + 8);
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] *= a.weight_offset + w[i];
        }
      }
      if (kind != 2 && turns_here) {
        const float4* cs = reinterpret_cast<const float4*>(s_cs + (buf * tpb + tl) * half + 8 * l);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 w = cs[i];
          const float p = x[2 * i], q = x[2 * i + 1], r = x[8 + 2 * i], s = x[9 + 2 * i];
          x[2 * i] = p * w.x - r * w.y, x[8 + 2 * i] = r * w.x + p * w.y;
          x[2 * i + 1] = q * w.z - s * w.w, x[9 + 2 * i] = s * w.z + q * w.w;
        }
      }
      auto put = [&](void* base_ptr, long long offset) {
        T* p = static_cast<T*>(base_ptr) + offset + first;
        store_vec<8>(p, x);
        store_vec<8>(p + second, x + 8);
      };
      if (kind == 0) put(a.q_out, t * a.q_out_stride + head * HD);
      if (kind == 1 && a.k_out != nullptr) put(a.k_out, t * a.k_out_stride + head * HD);
      if (kind == 1 && cache) put(a.k_cache, (row + head * 16) * HD);
      if (kind == 2) put(a.v_cache, (row + head * 16) * HD);
    }
    now = next;
    t += tpb;
    __syncthreads();
  }
}

template <typename T, int HD>
cudaError_t go(const QkRopeArgs& a, const Turns& turns, cudaStream_t s) {
  constexpr int L = HD / 16;
  const int items = a.Hq + (a.k_cache != nullptr ? 2 : 1) * a.Hkv;
  const int ipb = items < 512 / L ? items : 512 / L;
  int tpb = 256 / (ipb * L);
  if (tpb < 1) tpb = 1;
  if (tpb > a.T) tpb = a.T;
  const int threads = (tpb * ipb * L + 31) / 32 * 32;
  const int groups = (items + ipb - 1) / ipb;
  const size_t smem = (size_t)2 * tpb * (a.rotary / 2) * sizeof(float2);
  // as many blocks as are resident at once, each a run of tokens
  int resident = 2048 / threads;
  if (resident > 8) resident = 8;
  long long blocks = (long long)device_sm_count() * resident / groups;
  const long long rows = ((long long)a.T + tpb - 1) / tpb;
  if (blocks > rows) blocks = rows;
  if (blocks < 1) blocks = 1;
  const int per_block = (int)((rows + blocks - 1) / blocks) * tpb;
  const dim3 grid((unsigned)(((long long)a.T + per_block - 1) / per_block), groups);
  qk_rope_kernel<T, HD><<<grid, threads, smem, s>>>(a, turns, ipb, tpb, per_block);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkRopeArgs& a, cudaStream_t s) {
  if (a.cu != nullptr) {
    const PagedCheck c{a.cu, a.prefix_len, a.live, a.k_cache != nullptr ? a.block_table : nullptr,
                       a.B, a.T, a.T, a.max_blocks, a.num_blocks, -1, 0};
    const cudaError_t e = launch_paged_check(c, a.err, s);
    if (e != cudaSuccess) return e;
  }
  if (a.T == 0) return cudaSuccess;
  Turns turns;
  for (int c = 0; c < a.rotary / 2; ++c)
    turns.f[c] = (unsigned long long)ldexp(pow((double)a.theta, -2.0 * c / a.rotary) / 6.283185307179586476925286766559, 64);
  if (a.io == TV_F32) {
    if (a.hd == 64) return go<float, 64>(a, turns, s);
    return a.hd == 128 ? go<float, 128>(a, turns, s) : go<float, 256>(a, turns, s);
  }
  if (a.hd == 64) return go<bf16, 64>(a, turns, s);
  return a.hd == 128 ? go<bf16, 128>(a, turns, s) : go<bf16, 256>(a, turns, s);
}

}  // namespace tv
