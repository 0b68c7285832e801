// Norms of queries and keys per head, their rotation by position, and the new keys and values into the paged cache.
//
// y = x / sqrt(mean(x^2) + eps) * (offset + w) over a head's hd columns, then pairs (y_c, y_{c + r/2}), c < r/2, turned
// by position * theta^(-2c/r).  HD / 16 lanes take a head, each two vectors of eight columns that lie r/2 apart, so
// that a pair meets in one thread; columns past r come as two neighbouring vectors.
//
// Angles: theta^(-2c/r) / 2 pi is a fraction of a turn for each position.  In 64-bit fixed point position times that
// fraction drops whole turns by its overflow, exactly, however far the position; the nearest quarter turn comes off as
// two bits and what is left, an eighth of a turn at most, goes to sincospi rounded to 24 bits, 2^-28 of a turn.  The fraction
// is right to half of 2^-64 (tv_turns.h), so a position of 2^31 adds 2^-34 to that.  Angles are made once
// a token, eight tokens at a time by the whole block: made a token at a time by two warps, the others waited for them.
//
// Bound by HBM: q, k and v are read once and written once.  A block walks a run of tokens, its place among the sequences
// searched once, then counted on.  A thread's own vectors come through shared memory three tokens ahead, so that what is on
// its way does not lie in registers; no other thread reads them, and no barrier stands between.
//
// 14000 tokens, 32 + 8 + 8 heads of 128 columns: 344 MB in 63 us, 0.80 of the copy rate with 62 % of the issue slots taken; 64
// tokens behind a decode step 4.5 us.
#include "paged_check.cuh"
#include "tv_async.cuh"
#include "tv_common.cuh"
#include "tv_internal.h"
#include "tv_launch.cuh"
#include "tv_turns.h"

namespace tv {
namespace {

struct Turns {
  unsigned long long f[128];  // turns a position, in 2^-64
};

constexpr int kChunk = 8;  // tokens whose places and angles are made at a time, by the whole block
constexpr int kShared = 200 * 1024;  // of an SM for its blocks; one takes 147 KB at most (fp32, hd 256, 32 heads a block)
constexpr int kAhead = 4;  // tokens of a thread's vectors on their way, the one in work among them

// Sixteen columns as pairs of neighbours: eight from the first vector, eight from the second.
struct Columns {
  float2 x[8];
};
__device__ __forceinline__ void widen(uint4 v, float2* o) {
  o[0] = make_float2(bf16lo(v.x), bf16hi(v.x)), o[1] = make_float2(bf16lo(v.y), bf16hi(v.y));
  o[2] = make_float2(bf16lo(v.z), bf16hi(v.z)), o[3] = make_float2(bf16lo(v.w), bf16hi(v.w));
}
// A thread's vectors lie in shared memory 16 bytes a thread, so that neighbours' accesses meet all banks.
template <typename T>
struct Own;
template <>
struct Own<bf16> {
  static constexpr int kParts = 2;  // of 16 bytes
  template <typename P>
  __device__ static P* at(P* p, int part, int second) { return p + part * second; }
  __device__ static void widen16(const uint4* s, int step, Columns& c) { widen(s[0], c.x), widen(s[step], c.x + 4); }
};
template <>
struct Own<float> {
  static constexpr int kParts = 4;
  template <typename P>
  __device__ static P* at(P* p, int part, int second) { return p + (part / 2) * second + (part % 2) * 4; }
  __device__ static void widen16(const uint4* s, int step, Columns& c) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint4 v = s[k * step];
      c.x[2 * k] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
      c.x[2 * k + 1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
    }
  }
};

// tpb tokens side by side, ipb heads (queries, keys, and with a cache values) of each; per_block tokens a block.
template <typename T, int HD>
__global__ void __launch_bounds__(512, 2)
    qk_rope_kernel(const __grid_constant__ QkRopeArgs a, const __grid_constant__ Turns turns, int ipb, int tpb,
                   int per_block) {
  constexpr int L = HD / 16;
  constexpr int kParts = Own<T>::kParts;
  // the threads' vectors [kAhead][kParts][threads]; (cos, sin) of a chunk and the next [2][chunk][rotary / 2]; places of a
  // chunk and the next two [3][chunk]: position (-1: nothing to do) and block; the heads' weights
  extern __shared__ uint4 s_own[];
  const int half = a.rotary / 2;
  const int rounds = tpb < kChunk ? kChunk / tpb : 1, chunk = rounds * tpb;
  float2* s_cs = reinterpret_cast<float2*>(s_own + kAhead * kParts * blockDim.x);
  int2* s_place = reinterpret_cast<int2*>(s_cs + 2 * chunk * half);
  float2* s_w = reinterpret_cast<float2*>(s_place + 3 * chunk + (chunk & 1));  // offset + weight, of queries and of keys: [2][8][L]
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

  // columns first .. first + 7, and as many `second` further on
  const bool turns_here = l < a.rotary / 16;
  const int first = turns_here ? 8 * l : a.rotary + 16 * (l - a.rotary / 16);
  const int second = turns_here ? half : 8;
  const long long x_stride = (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) * tpb;
  int t = (int)t0 + tl;
  const T* from = static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) + t * (x_stride / tpb) + head * HD + first;

  // Copies need no place among the sequences: they go ahead of everything.  copied: the token that is copied next.
  int copied = mine ? t : 0x7fffffff, to_stage = 0;
  auto copy = [&]() {
    if (copied < t1) {
#pragma unroll
      for (int i = 0; i < kParts; ++i)
        cp_async_16_cg(s_own + (to_stage * kParts + i) * blockDim.x + threadIdx.x, Own<T>::at(from, i, second));
      from += x_stride;
      copied = copied < 0x7fffffff - tpb ? copied + tpb : 0x7fffffff;
    }
    to_stage = to_stage + 1 == kAhead ? 0 : to_stage + 1;
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < kAhead - 1; ++k) copy();

  const bool scaled = a.norm && kind != 2;
  const bool weighted = a.norm && (kind == 0 ? a.q_weight != nullptr : kind == 1 && a.k_weight != nullptr);
  for (int i = threadIdx.x; i < 2 * HD; i += blockDim.x) {
    const T* w = static_cast<const T*>(i < HD ? a.q_weight : a.k_weight);
    if (w == nullptr) continue;
    // column c of a head is its lane's l place e: as in first and second
    const int c = i % HD;
    int lane, e;
    if (c < half) lane = c / 8, e = c % 8;
    else if (c < 2 * half) lane = (c - half) / 8, e = 8 + (c - half) % 8;
    else lane = half / 8 + (c - 2 * half) / 16, e = (c - 2 * half) % 16;
    reinterpret_cast<float*>(s_w + (i / HD * 8 + e / 2) * L + lane)[e % 2] = a.weight_offset + to_f32(w[c]);
  }

  wait_for_plan();
  // Thread i < chunk follows the i-th token of each chunk: its sequence (-1: before the first, B: past the last), the token
  // past its last, what to add to a token's number for its position.
  int b = -1, end = 0, shift = 0;
  bool open = false;  // the sequence's tokens are worked on
  if (a.cu != nullptr) {
    if (a.err[0] == TV_ERR_BAD_SEQLEN) {
      cp_async_wait<0>();
      return;
    }
    // the sequences that end at or before the block's first token lie behind it
    int n = 0;
    for (int i = threadIdx.x % 32; i <= a.B; i += 32) n += a.cu[i] <= t0;
    n = __reduce_add_sync(0xffffffffu, n);
    b = n - 2;  // find() enters the sequence itself
    end = n > 0 ? (int)t0 : a.cu[0];
  }
  auto find = [&](int token) -> int2 {  // tokens come in ascending order
    if (a.cu != nullptr) {
      while (b < a.B && token >= end) {
        ++b;
        end = b < a.B ? a.cu[b + 1] : 0x7fffffff;
        open = false;
        if (b >= 0 && b < a.B && token < end) {
          shift = (a.prefix_len != nullptr ? a.prefix_len[b] : 0) - a.cu[b];
          open = a.err[b] == 0 && (a.live == nullptr || a.live[b] != 0);
        }
      }
      if (!open) return make_int2(-1, 0);
      const int position = token + shift;
      return make_int2(position, cache ? a.block_table[(long long)b * a.max_blocks + position / 16] : 0);
    }
    // one token a sequence: checked here
    int st = 0, block = 0;
    const bool live = a.live == nullptr || a.live[token] != 0;
    const int position = a.prefix_len != nullptr ? a.prefix_len[token] : 0;
    if (live && (position < 0 || position >= (cache ? a.max_blocks * 16 : 0x7fffffff))) st = TV_ERR_CAPACITY;
    if (live && st == 0 && cache) {
      block = a.block_table[(long long)token * a.max_blocks + position / 16];
      if ((unsigned)block >= (unsigned)a.num_blocks) st = TV_ERR_BAD_BLOCK;
    }
    if (blockIdx.y == 0) a.err[token] = st;
    return make_int2(live && st == 0 ? position : -1, block);
  };
  auto places = [&](int k) {  // of chunk k
    const int i = threadIdx.x;
    const long long token = t0 + (long long)k * chunk + i;
    if (i < chunk) s_place[k % 3 * chunk + i] = token < t1 ? find((int)token) : make_int2(-1, 0);
  };
  // Pair i = 0 .. 3 of lane l's eight columns lies at [i][l], so that a head's lanes read side by side.
  auto angles = [&](int k) {
    for (int i = threadIdx.x; i < chunk * half; i += blockDim.x) {
      const int token = i / half, c = i - token * half;
      const int position = s_place[k % 3 * chunk + token].x;
      if (position < 0) continue;
      const unsigned long long turn = (unsigned long long)(unsigned)position * turns.f[c];
      const unsigned long long quarter = (turn + (1ull << 61)) >> 62;
      const int rest = (int)((long long)(turn - (quarter << 62)) >> 30);  // in 2^-34 of a turn
      float sn, cn;
      sincospif((float)rest * 0x1p-33f, &sn, &cn);
      const float2 even = make_float2(cn, sn), odd = make_float2(-sn, cn);
      float2 v = quarter & 1 ? odd : even;
      if (quarter & 2) v.x = -v.x, v.y = -v.y;
      // as two cosines and two sines: registers that lie side by side
      float* to = reinterpret_cast<float*>(s_cs + ((k & 1) * chunk + token) * half + (c % 8 / 2 * (half / 8) + c / 8) * 2) + c % 2;
      to[0] = v.x, to[2] = v.y;
    }
  };

  places(0);
  places(1);
  __syncthreads();
  angles(0);
  T* q_to = static_cast<T*>(a.q_out) + t * a.q_out_stride + head * HD + first;
  T* k_to = a.k_out != nullptr ? static_cast<T*>(a.k_out) + t * a.k_out_stride + head * HD + first : nullptr;
  int round = 0, chunk_at = 0, stage = 0;
  const float2* w_own = s_w + (kind * 8) * L + l;
  for (int base = (int)t0; base < t1; base += tpb) {
    if (round == 0) {  // this chunk's angles are there, the last one's are done with
      __syncthreads();
      places(chunk_at + 2);
      angles(chunk_at + 1);
    }
    copy();
    const int in_chunk = round * tpb + tl;
    const int2 place = mine ? s_place[chunk_at % 3 * chunk + in_chunk] : make_int2(-1, 0);
    const bool now = place.x >= 0;
    cp_async_wait<kAhead - 1>();
    const uint4* own = s_own + stage * kParts * blockDim.x + threadIdx.x;
    stage = stage + 1 == kAhead ? 0 : stage + 1;
    const long long row = (((long long)place.y * a.Hkv + head) * 16 + (place.x & 15)) * HD + first;
    Columns c;
    float2 sum2 = make_float2(0.f, 0.f);
    if (now && kind != 2) {
      Own<T>::widen16(own, blockDim.x, c);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum2 = __ffma2_rn(c.x[i], c.x[i], sum2);
    }
    const float sum = group_sum<L>(sum2.x + sum2.y);
    if (now && kind != 2) {
      if (scaled) {
        const float inv = rsqrtf(sum / HD + a.eps);
        const float2 inv2 = make_float2(inv, inv);
#pragma unroll
        for (int i = 0; i < 8; ++i) c.x[i] = __fmul2_rn(c.x[i], inv2);
        if (weighted)
#pragma unroll
          for (int i = 0; i < 8; ++i) c.x[i] = __fmul2_rn(c.x[i], w_own[i * L]);
      }
      if (turns_here) {
        const float4* cs = reinterpret_cast<const float4*>(s_cs + ((chunk_at & 1) * chunk + in_chunk) * half) + l;
        const float2 minus = make_float2(-1.f, -1.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 v = cs[i * (half / 8)];  // of two columns
          const float2 cos2 = make_float2(v.x, v.y), sin2 = make_float2(v.z, v.w);
          const float2 p = c.x[i], q = c.x[4 + i];
          c.x[i] = __ffma2_rn(p, cos2, __fmul2_rn(__fmul2_rn(q, sin2), minus));
          c.x[4 + i] = __ffma2_rn(p, sin2, __fmul2_rn(q, cos2));
        }
      }
      auto put = [&](T* p) {
        store_vec<8>(p, &c.x[0].x);
        store_vec<8>(p + second, &c.x[4].x);
      };
      if (kind == 0) {
        put(q_to);
      } else {
        if (a.k_out != nullptr) put(k_to);
        if (cache) put(static_cast<T*>(a.k_cache) + row);
      }
    } else if (now) {
      // a value goes as it is
#pragma unroll
      for (int i = 0; i < kParts; ++i)
        *reinterpret_cast<uint4*>(Own<T>::at(static_cast<T*>(a.v_cache) + row, i, second)) = own[i * blockDim.x];
    }
    q_to += a.q_out_stride * tpb;
    if (a.k_out != nullptr) k_to += a.k_out_stride * tpb;
    if (++round == rounds) round = 0, ++chunk_at;
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
  const int chunk = tpb < kChunk ? kChunk / tpb * tpb : tpb;
  const size_t smem = (size_t)kAhead * Own<T>::kParts * threads * 16 + (size_t)chunk * (a.rotary * sizeof(float2) + 3 * sizeof(int2)) + 8 + 2 * HD * sizeof(float);
  auto kern = qk_rope_kernel<T, HD>;
  // One limit for all shapes: with each call's own, another thread's call might lower it before this one's launch.
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kShared);
    if (e != cudaSuccess) return e;
  }
  // as many blocks as are resident at once (64 registers a thread), each a run of tokens
  int resident = 1024 / threads;
  if (resident > (int)(kShared / smem)) resident = (int)(kShared / smem);
  if (resident < 1) resident = 1;
  long long blocks = (long long)device_sm_count() * resident / groups;
  const long long rows = ((long long)a.T + tpb - 1) / tpb;
  if (blocks > rows) blocks = rows;
  if (blocks < 1) blocks = 1;
  const int per_block = (int)((rows + blocks - 1) / blocks) * tpb;
  const dim3 grid((unsigned)(((long long)a.T + per_block - 1) / per_block), groups);
  if (a.cu != nullptr) return launch_behind_plan(kern, grid, threads, smem, s, a, turns, ipb, tpb, per_block);
  kern<<<grid, threads, smem, s>>>(a, turns, ipb, tpb, per_block);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkRopeArgs& a, cudaStream_t s) {
  if (a.cu != nullptr) {
    const PagedCheck c{a.cu, a.prefix_len, a.live, a.k_cache != nullptr ? a.block_table : nullptr,
                       a.B, a.T, a.T, a.max_blocks, a.num_blocks, -1, 0, a.err};
    const cudaError_t e = launch_paged_check(c, s);
    if (e != cudaSuccess) return e;
  }
  if (a.T == 0) return cudaSuccess;
  Turns turns;
  turns_of(a.theta, a.rotary, turns.f);
  if (a.io == TV_F32) {
    if (a.hd == 64) return go<float, 64>(a, turns, s);
    return a.hd == 128 ? go<float, 128>(a, turns, s) : go<float, 256>(a, turns, s);
  }
  if (a.hd == 64) return go<bf16, 64>(a, turns, s);
  return a.hd == 128 ? go<bf16, 128>(a, turns, s) : go<bf16, 256>(a, turns, s);
}

}  // namespace tv
