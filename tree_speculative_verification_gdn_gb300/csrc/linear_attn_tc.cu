// Linear attention with a decay over prompts on the 5th-generation tensor cores (bf16 I/O).
//
// A prompt (or a segment of one) and head is walked in chunks of C = 128 tokens with the state on
// chip.  With g_i the log2 of the decay from before the chunk to token i, inclusive, and S the
// state before the chunk (dv x dk):
//     P_ij = 2^(g_i - g_j) q_scale q_i.k_j  (j <= i),       O = P V + diag(2^g q_scale) Q S^T,
//     S   <- 2^g_C S + V^T K',                              k'_j = 2^(g_C - g_j) k_j.
// Four products a chunk, all C x 128 x 128, operands in shared memory as TMA lays them (128-byte
// swizzle), accumulators and the state in the 512 columns of tensor memory:
//     QK: scores [token i, token j]      A = Q, B = K
//     QS: O_inter [token i, value]       A = Q, B = S          (bf16 pair)
//     ST: S [value, key column]          A = V^T, B = K'       (bf16 pair), added to the state
//     PV: O_intra [token i, value]       A = P (bf16 pair, tensor memory, over the scores), B = V
// P, K' and S are fp32 results and enter as value + remainder, two bf16 each (2^-16 left out): one
// bf16 alone would put an error as large as the output's own rounding on every output, and 2^-9 on
// an fp32 state.  Exponents only ever go down: within 32 x 32 diagonal blocks each 2^(g_i - g_j) is
// taken directly, elsewhere as 2^(g_i - g_r) 2^(g_r - g_j) with r the first row of i's block, so no
// factor exceeds 1 however fast the decay.  g is summed in 64 bits and kept as two floats: after a
// reset (alpha near 0) small differences of large sums remain.
//
// Twelve warps: four turn scores into P and write outputs (thread = token), four own the state
// (thread = value row) and scale the keys, one issues TMA loads, one the MMAs, one sums the decays.
// A ring of whole tiles (Q, K, V, Q, ...) feeds them; every tile is given back by the MMA that reads
// it last.  One CTA per SM, since the state, its bf16 pair and four 32 KB tiles fill shared memory.
#include "linear_attn.cuh"
#include "tv_async.cuh"
#include "tv_tc.cuh"
#include "tv_tma_host.h"

namespace tv {
namespace {

constexpr int kC = 128;         // tokens per chunk
constexpr int kThreads = 352;   // 4 + 4 warps, TMA, MMA and decay warps
constexpr int kHalf = kC * 128; // bytes of 64 columns of a 128-token tile
constexpr uint32_t kPolls = 1u << 18;
constexpr int kSmemMax = 232448;
constexpr int kMaxSlots = 8;

// TMEM columns
constexpr uint32_t kColQK = 0, kColS = 128, kColIntra = 256, kColInter = 384;

struct Shared {
  float2 g[2][kC];            // g_i as two floats, by chunk parity
  float f[192];               // 2^(g_r - g_j) of row blocks 1, 2, 3: 32, 64, 96 entries
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t g_full[2], g_empty[2];
  uint64_t qk_done, s_ready, k_ready, p_ready, st_done, o_done, o_free, drain;
  uint32_t tmem;
  int fail;
};

template <int DK, int DV, bool STATE_ONLY>
struct Plan {
  static constexpr int slot = kC * 2 * (DK > DV ? DK : DV);
  static constexpr int lo = kC * 2 * DK;                    // remainders of K'
  static constexpr int s = STATE_ONLY ? 0 : DV * DK * 2;    // the state's bf16 values; as much for its remainders
  static constexpr int room = kSmemMax - lo - 2 * s - (int)sizeof(Shared);
  static constexpr int slots = room / slot < kMaxSlots ? room / slot : kMaxSlots;
  static constexpr int bytes = slots * slot + lo + 2 * s + (int)sizeof(Shared);
  static_assert(slots >= 3, "a chunk's tiles fit");
};

__device__ __forceinline__ bool try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
// Waits for the phase of that parity; false once this or another warp has given up.
__device__ __forceinline__ bool wait(Shared& sh, uint64_t* bar, uint32_t parity) {
  for (uint32_t it = 0; it < kPolls; ++it) {
    if (try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&sh.fail)) return false;
  }
  *reinterpret_cast<volatile int*>(&sh.fail) = 1;
  return false;
}

// The same for a whole warp, one answer for all of it.
__device__ __forceinline__ bool wait_warp(Shared& sh, uint64_t* bar, uint32_t parity) {
  const bool ok = wait(sh, bar, parity);
  return __all_sync(0xffffffffu, ok);
}

// 32 columns of this thread's lane; tmem_join() before their first use.
__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t* r) {
  tmem_ld16_nowait(at, r);
  tmem_ld16_nowait(at + 16, r + 16);
}
template <int N>
__device__ __forceinline__ void tmem_join(uint32_t* r) {
#pragma unroll
  for (int k = 0; k < N; ++k) asm volatile("" : "+r"(r[k]));
}
// 16 columns, without the wait.
__device__ __forceinline__ void tmem_st16_nowait(uint32_t at, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// x as value and remainder, two columns a word.
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(x0, x1);
  lo = pack_bf16x2(x0 - bf16lo(hi), x1 - bf16hi(hi));
}

__device__ __forceinline__ float exp2_gap(float2 a, float2 b) { return exp2f((a.x - b.x) + (a.y - b.y)); }

constexpr uint32_t kIdescAMn = 1u << 15;  // A with its M dimension contiguous

template <int DK, int DV, typename TST, bool STATE_ONLY>
__global__ void __launch_bounds__(kThreads, 1)
    linear_attn_tc_kernel(const __grid_constant__ LinAttnArgs a, int units, const __grid_constant__ CUtensorMap mq,
                          const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using L = Plan<DK, DV, STATE_ONLY>;
  constexpr int kTiles = STATE_ONLY ? 2 : 3;  // tiles per chunk: (Q,) K, V
  constexpr int kK = kTiles - 2, kV = kTiles - 1;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* s_lo = smem + L::slots * L::slot;
  unsigned char* s_hi = s_lo + L::lo;  // state values, then their remainders
  Shared& sh = *reinterpret_cast<Shared*>(s_hi + 2 * L::s);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

  const bool ok = check_seqlens(a);
  if (blockIdx.x == 0 && (STATE_ONLY || a.seg_len == 0))
    for (int b = tid; b < a.B; b += kThreads) a.err[b] = ok ? 0 : TV_ERR_BAD_SEQLEN;
  if (!ok) return;

  if (tid == 0) {
    for (int i = 0; i < L::slots; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.g_full[i], 1);
      mbar_init(&sh.g_empty[i], STATE_ONLY ? 4 : 8);
    }
    mbar_init(&sh.qk_done, 1);
    mbar_init(&sh.s_ready, 128);
    mbar_init(&sh.k_ready, 128);
    mbar_init(&sh.p_ready, 128);
    mbar_init(&sh.st_done, 1);
    mbar_init(&sh.o_done, 1);
    mbar_init(&sh.o_free, 128);
    mbar_init(&sh.drain, 1);
    sh.fail = 0;
    mbar_fence_init();
  }
  if (warp == 9) tmem_alloc(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  // Every role walks the same units and chunks; n counts chunks over all units, m tiles.
  int n = 0;
  bool good = true;
  if (warp < 4) {
    // ------------------------------------------------ scores to P, outputs (thread = token)
    if constexpr (!STATE_ONLY) {
      const uint32_t row = tmem + ((uint32_t)(32 * warp) << 16);
      float* f = sh.f + (warp == 2 ? 32 : warp == 3 ? 96 : 0);  // 32 * warp entries
      for (int u = blockIdx.x; u < units && good; u += gridDim.x) {
        const Segment seg = find_segment(a, u / a.H);
        if (seg.b < 0) break;
        bf16* out = static_cast<bf16*>(a.out) + (long long)(u % a.H) * DV;
        for (int t = seg.t0; t < seg.t1; t += kC, ++n) {
          const float2* g = sh.g[n & 1];
          if (!(good = wait_warp(sh, &sh.g_full[n & 1], (n >> 1) & 1))) break;
          const float2 gi = g[tid], gr = g[32 * warp];
          const float into = exp2f(gi.x + gi.y) * a.q_scale;  // of the state before the chunk
          const float ei = exp2_gap(gi, gr) * a.q_scale;
          __syncwarp();  // the last chunk's readers of f are done
          for (int p = 0; p < warp; ++p) f[lane + 32 * p] = exp2_gap(gr, g[lane + 32 * p]);
          __syncwarp();
          if (!(good = wait_warp(sh, &sh.qk_done, n & 1))) break;
          tc_fence_after();
          // P of columns 32 p .. + 31: values to columns 16 p, remainders to 64 + 16 p, over scores
          // already read; remainders wait in registers for that.
          uint32_t lo[4][16];
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            uint32_t s[32], hi[16];
            if (p > warp) {
#pragma unroll
              for (int c = 0; c < 16; ++c) hi[c] = lo[p][c] = 0;
            } else {
              tmem_ld32(row + kColQK + 32 * p, s);
              tmem_wait_ld();
              tmem_join<32>(s);
              float x[32];
              if (p < warp) {
#pragma unroll
                for (int c = 0; c < 32; c += 4) {
                  const float4 fj = *reinterpret_cast<const float4*>(f + 32 * p + c);
                  x[c] = __uint_as_float(s[c]) * fj.x * ei;
                  x[c + 1] = __uint_as_float(s[c + 1]) * fj.y * ei;
                  x[c + 2] = __uint_as_float(s[c + 2]) * fj.z * ei;
                  x[c + 3] = __uint_as_float(s[c + 3]) * fj.w * ei;
                }
              } else {
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                  const float e = exp2_gap(gi, g[32 * p + c]) * a.q_scale;
                  x[c] = c <= lane ? __uint_as_float(s[c]) * e : 0.f;
                }
              }
#pragma unroll
              for (int c = 0; c < 16; ++c) split2(x[2 * c], x[2 * c + 1], hi[c], lo[p][c]);
            }
            tmem_st16_nowait(row + kColQK + 16 * p, hi);
          }
#pragma unroll
          for (int p = 0; p < 4; ++p) tmem_st16_nowait(row + kColQK + 64 + 16 * p, lo[p]);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&sh.p_ready);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.g_empty[n & 1]);
          if (!(good = wait_warp(sh, &sh.o_done, n & 1))) break;
          tc_fence_after();
          bf16* o = out + (t + tid) * a.out_stride;
#pragma unroll
          for (int c = 0; c < DV; c += 32) {
            uint32_t x[32], y[32];
            tmem_ld32(row + kColInter + c, x);
            tmem_ld32(row + kColIntra + c, y);
            tmem_wait_ld();
            tmem_join<32>(x);
            tmem_join<32>(y);
            if (c + 32 == DV) {
              tc_fence_before();
              mbar_arrive(&sh.o_free);
            }
            if (t + tid < seg.t1) {
              float z[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) z[i] = fmaf(into, __uint_as_float(x[i]), __uint_as_float(y[i]));
              store_vec<32>(o + c, z);
            }
          }
        }
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------ the state (thread = value row) and K'
    const int r = tid - 128;
    const uint32_t row = tmem + ((uint32_t)(32 * (warp - 4)) << 16) + kColS;
    const bool mine = 32 * (warp - 4) < DV;  // warp-uniform
    for (int u = blockIdx.x; u < units && good; u += gridDim.x) {
      const Segment seg = find_segment(a, u / a.H);
      if (seg.b < 0) break;
      const bool last = seg.index + 1 == seg.count;
      if (STATE_ONLY && last) continue;
      const size_t head = ((size_t)seg.b * a.H + u % a.H) * DV * DK + r * DK, slot = (size_t)u * DV * DK + r * DK;
      float total = 1.f;
      if (mine) {
#pragma unroll
        for (int c = 0; c < DK; c += 16) {
          float x[16];
          if (!STATE_ONLY && seg.count > 1) {
            load_vec_rw<16>(a.slots + slot + c, x);
          } else if (!STATE_ONLY && a.S0 != nullptr) {
            load_vec_rw<16>(static_cast<const TST*>(a.S0) + head + c, x);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = 0.f;
          }
          tmem_st16_nowait(row + c, reinterpret_cast<const uint32_t*>(x));
        }
        tmem_wait_st();
      }
      for (int t = seg.t0; t < seg.t1; t += kC, ++n) {
        const float2* g = sh.g[n & 1];
        if (!(good = wait_warp(sh, &sh.g_full[n & 1], (n >> 1) & 1))) break;
        if (t > seg.t0 && !(good = wait_warp(sh, &sh.st_done, (n - 1) & 1))) break;
        tc_fence_after();
        const float2 gc = g[kC - 1];
        const float keep = exp2f(gc.x + gc.y);
        if (STATE_ONLY) total *= keep;
        if (mine) {
#pragma unroll
          for (int c = 0; c < DK; c += 32) {
            uint32_t s[32];
            tmem_ld32(row + c, s);
            tmem_wait_ld();
            tmem_join<32>(s);
            if (!STATE_ONLY) {
              unsigned char* to = s_hi + (c / 64) * (DV * 128) + r * 128;
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                uint4 hi, lo;
                split2(__uint_as_float(s[8 * v]), __uint_as_float(s[8 * v + 1]), hi.x, lo.x);
                split2(__uint_as_float(s[8 * v + 2]), __uint_as_float(s[8 * v + 3]), hi.y, lo.y);
                split2(__uint_as_float(s[8 * v + 4]), __uint_as_float(s[8 * v + 5]), hi.z, lo.z);
                split2(__uint_as_float(s[8 * v + 6]), __uint_as_float(s[8 * v + 7]), hi.w, lo.w);
                const int at = ((c % 64 / 8 + v) ^ (r & 7)) * 16;
                *reinterpret_cast<uint4*>(to + at) = hi;
                *reinterpret_cast<uint4*>(to + L::s + at) = lo;
              }
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) s[i] = __float_as_uint(__uint_as_float(s[i]) * keep);
            tmem_st16_nowait(row + c, s);
            tmem_st16_nowait(row + c + 16, s + 16);
          }
          tmem_wait_st();
        }
        fence_proxy_async();
        tc_fence_before();
        mbar_arrive(&sh.s_ready);
        // Keys: 16 bytes at a time where TMA left them, row j = (tid / 8 + 16 i) % 128.  Rows past the
        // segment's end hold another prompt's tokens, or none: K' and V rows there become zero.
        const int m = n * kTiles, ks = (m + kK) % L::slots;
        const int rows = seg.t1 - t;
        float scale[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) scale[i] = exp2_gap(gc, g[r / 8 + 16 * i]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.g_empty[n & 1]);
        if (!(good = wait_warp(sh, STATE_ONLY ? &sh.full[ks] : &sh.qk_done, STATE_ONLY ? ((m + kK) / L::slots) & 1 : n & 1)))
          break;
        if (rows < kC) {
          const int vs = (m + kV) % L::slots;
          if (!(good = wait_warp(sh, &sh.full[vs], ((m + kV) / L::slots) & 1))) break;
          for (int i = r; i < kC * DV / 8; i += 128)
            if (i / 8 % kC >= rows) reinterpret_cast<uint4*>(smem + vs * L::slot)[i] = make_uint4(0, 0, 0, 0);
        }
        uint4* kt = reinterpret_cast<uint4*>(smem + ks * L::slot);
        uint4* lt = reinterpret_cast<uint4*>(s_lo);
        for (int half = 0; half < DK / 64; ++half)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int at = (half * 8 + i) * 128 + r;
            float x[8];
            unpack8(kt[at], x);
            const bool in = r / 8 + 16 * i < rows;
#pragma unroll
            for (int c = 0; c < 8; ++c) x[c] = in ? x[c] * scale[i] : 0.f;
            uint4 hi, lo;
            split2(x[0], x[1], hi.x, lo.x);
            split2(x[2], x[3], hi.y, lo.y);
            split2(x[4], x[5], hi.z, lo.z);
            split2(x[6], x[7], hi.w, lo.w);
            kt[at] = hi;
            lt[at] = lo;
          }
        fence_proxy_async();
        mbar_arrive(&sh.k_ready);
      }
      if (!good) break;
      if (seg.t1 > seg.t0) {
        if (!(good = wait_warp(sh, &sh.st_done, (n - 1) & 1))) break;
        tc_fence_after();
      }
      if (mine && (STATE_ONLY || last)) {
#pragma unroll
        for (int c = 0; c < DK; c += 32) {
          uint32_t s[32];
          tmem_ld32(row + c, s);
          tmem_wait_ld();
          tmem_join<32>(s);
          if (STATE_ONLY) store_vec<32>(a.slots + slot + c, reinterpret_cast<const float*>(s));
          else store_vec<32>(static_cast<TST*>(a.S) + head + c, reinterpret_cast<const float*>(s));
        }
      }
      if (STATE_ONLY && r == 0) a.decay[u] = total;
    }
  } else if (warp == 8) {
    // ------------------------------------------------ TMA loads
    int m = 0;
    for (int u = blockIdx.x; u < units && good; u += gridDim.x) {
      const Segment seg = find_segment(a, u / a.H);
      if (seg.b < 0) break;
      if (STATE_ONLY && seg.index + 1 == seg.count) continue;
      const int h = u % a.H, hk = h / (a.H / a.Hk);
      if (lane == 0) {
        for (int t = seg.t0; t < seg.t1 && good; t += kC) {
          for (int tile = 0; tile < kTiles; ++tile, ++m) {
            const int s = m % L::slots;
            if (m >= L::slots && !(good = wait(sh, &sh.empty[s], (m / L::slots - 1) & 1))) break;
            const bool is_v = tile == kV;
            const int halves = (is_v ? DV : DK) / 64;
            mbar_arrive_expect_tx(&sh.full[s], halves * kHalf);
            const CUtensorMap* map = is_v ? &mv : tile == kK ? &mk : &mq;
            for (int x = 0; x < halves; ++x)
              tma_load_3d(smem + s * L::slot + x * kHalf, map, 64 * x, is_v ? h : hk, t, &sh.full[s]);
          }
        }
      }
      good = __shfl_sync(0xffffffffu, good, 0);
    }
    if (!good && lane == 0)  // leave no copy in flight behind
      for (int i = m > L::slots ? m - L::slots : 0; i < m; ++i)
        mbar_wait(&sh.full[i % L::slots], (i / L::slots) & 1);
  } else if (warp == 9) {
    // ------------------------------------------------ MMAs
    for (int u = blockIdx.x; u < units && good; u += gridDim.x) {
      const Segment seg = find_segment(a, u / a.H);
      if (seg.b < 0) break;
      if (STATE_ONLY && seg.index + 1 == seg.count) continue;
      if (lane == 0) {
        for (int t = seg.t0; t < seg.t1; t += kC, ++n) {
          const int m = n * kTiles;
          const int qs = m % L::slots, ks = (m + kK) % L::slots, vs = (m + kV) % L::slots;
          const uint32_t q = smem_addr(smem + qs * L::slot), k = smem_addr(smem + ks * L::slot),
                         v = smem_addr(smem + vs * L::slot), lo = smem_addr(s_lo), st = smem_addr(s_hi);
          if (!STATE_ONLY) {
            if (!(good = wait(sh, &sh.full[qs], (m / L::slots) & 1))) break;
            if (!(good = wait(sh, &sh.full[ks], ((m + kK) / L::slots) & 1))) break;
            tc_fence_after();
            constexpr uint32_t id = idesc_bf16_f32(kC, kC);
            for (int c = 0; c < DK; c += 16) {
              const uint32_t at = c / 64 * kHalf + c % 64 * 2;
              mma_bf16(tmem + kColQK, sw128_desc(q + at), sw128_desc(k + at), id, c > 0);
            }
            mma_commit(&sh.qk_done);
            if (!(good = wait(sh, &sh.s_ready, n & 1))) break;
            if (n > 0 && !(good = wait(sh, &sh.o_free, (n - 1) & 1))) break;
            tc_fence_after();
            constexpr uint32_t ids = idesc_bf16_f32(kC, DV);
            for (int part = 0; part < 2; ++part)
              for (int c = 0; c < DK; c += 16)
                mma_bf16(tmem + kColInter, sw128_desc(q + c / 64 * kHalf + c % 64 * 2),
                         sw128_desc(st + part * L::s + c / 64 * (DV * 128) + c % 64 * 2), ids, part + c > 0);
            mma_commit(&sh.empty[qs]);
          } else if (!(good = wait(sh, &sh.s_ready, n & 1))) {
            break;
          }
          if (!(good = wait(sh, &sh.k_ready, n & 1))) break;
          if (!(good = wait(sh, &sh.full[vs], ((m + kV) / L::slots) & 1))) break;
          tc_fence_after();
          // M = 128 value rows; with dv = 64 the upper 64 read what lies behind the tile and land in
          // tensor-memory lanes that nobody reads.
          constexpr uint32_t idt = idesc_bf16_f32(kC, DK, true) | kIdescAMn;
          for (int part = 0; part < 2; ++part)
            for (int c = 0; c < kC; c += 16)
              mma_bf16(tmem + kColS, sw128_mn_desc(v + c * 128, kHalf), sw128_mn_desc((part ? lo : k) + c * 128, kHalf),
                       idt, 1);
          mma_commit(&sh.st_done);
          mma_commit(&sh.empty[ks]);
          if (STATE_ONLY) {
            mma_commit(&sh.empty[vs]);
          } else {
            if (!(good = wait(sh, &sh.p_ready, n & 1))) break;
            tc_fence_after();
            constexpr uint32_t idp = idesc_bf16_f32(kC, DV, true);
            for (int part = 0; part < 2; ++part)
              for (int c = 0; c < kC; c += 16)
                mma_bf16_tmem_a(tmem + kColIntra, tmem + kColQK + 64 * part + c / 2,
                                sw128_mn_desc(v + c * 128, kHalf), idp, part + c > 0);
            mma_commit(&sh.o_done);
            mma_commit(&sh.empty[vs]);
          }
        }
      }
      good = __shfl_sync(0xffffffffu, good, 0);
      n = __shfl_sync(0xffffffffu, n, 0);
    }
  } else {
    // ------------------------------------------------ decays: lane l sums tokens 4 l .. 4 l + 3
    for (int u = blockIdx.x; u < units && good; u += gridDim.x) {
      const Segment seg = find_segment(a, u / a.H);
      if (seg.b < 0) break;
      if (STATE_ONLY && seg.index + 1 == seg.count) continue;
      const float* al = a.alpha + u % a.H;
      for (int t = seg.t0; t < seg.t1; t += kC, ++n) {
        double sum[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = t + 4 * lane + i;
          const float x = tok < seg.t1 ? __ldg(al + tok * a.alpha_stride) : 1.f;
          // alpha = 0 forgets everything: 2^-1000 times any state is 0 in fp32
          sum[i] = x == 0.f ? -1000.f : log2f(x);
          if (i > 0) sum[i] += sum[i - 1];
        }
        double up = sum[3];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double below = __shfl_up_sync(0xffffffffu, up, o);
          if (lane >= o) up += below;
        }
        up -= sum[3];
        if (n >= 2 && !(good = wait_warp(sh, &sh.g_empty[n & 1], ((n >> 1) - 1) & 1))) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const double x = up + sum[i];
          const float hi = (float)x;
          sh.g[n & 1][4 * lane + i] = make_float2(hi, (float)(x - hi));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.g_full[n & 1]);
      }
    }
  }
  __syncwarp();
  // Every MMA has completed: the state's owners waited for the last of each unit, the outputs' for
  // theirs; after a wait that gave up the last ones issued may still run, so wait for them too.
  if (warp == 9 && lane == 0 && *reinterpret_cast<volatile int*>(&sh.fail)) {
    mma_commit(&sh.drain);
    mbar_wait(&sh.drain, 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) tmem_dealloc(tmem, 512);
  if (sh.fail && warp == 0)
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
      const Segment seg = find_segment(a, u / a.H);
      if (seg.b < 0) break;
      if (lane == 0) a.err[seg.b] = TV_ERR_TIMEOUT;
    }
}

// [T, heads, d] with a token stride: boxes of 64 columns of one head and 128 tokens; tokens past
// the end read as zero.
bool token_map(CUtensorMap* m, const void* p, int d, int heads, int T, long long stride) {
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, 1, kC};
  return make_map_bf16_sw128(m, p, 3, dims, strides, box);
}

template <int DK, int DV, typename TST, bool STATE_ONLY>
cudaError_t go(const LinAttnArgs& a, int units, const CUtensorMap* m, cudaStream_t s) {
  using L = Plan<DK, DV, STATE_ONLY>;
  auto* fn = linear_attn_tc_kernel<DK, DV, TST, STATE_ONLY>;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, L::bytes);
  if (e != cudaSuccess) return e;
  const int sms = device_sm_count();
  fn<<<units < sms ? units : sms, kThreads, L::bytes, s>>>(a, units, m[0], m[1], m[2]);
  return cudaGetLastError();
}

template <int DK, int DV, typename TST>
cudaError_t prompt_tc(const LinAttnArgs& a, cudaStream_t s) {
  CUtensorMap m[3];
  if (!token_map(&m[0], a.q, DK, a.Hk, a.T, a.q_stride) || !token_map(&m[1], a.k, DK, a.Hk, a.T, a.k_stride) ||
      !token_map(&m[2], a.v, DV, a.H, a.T, a.v_stride))
    return cudaErrorInvalidValue;
  const long long units = (a.seg_len > 0 ? (long long)a.B + a.T / a.seg_len : a.B) * a.H;
  if (units > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (a.seg_len > 0) {
    cudaError_t e = go<DK, DV, TST, true>(a, (int)units, m, s);
    if (e == cudaSuccess) e = launch_linear_attn_scan(a, s);
    if (e != cudaSuccess) return e;
  }
  return go<DK, DV, TST, false>(a, (int)units, m, s);
}

template <typename TST>
cudaError_t prompt_dims(const LinAttnArgs& a, cudaStream_t s) {
  if (a.dk == 64) return a.dv == 64 ? prompt_tc<64, 64, TST>(a, s) : prompt_tc<64, 128, TST>(a, s);
  return a.dv == 64 ? prompt_tc<128, 64, TST>(a, s) : prompt_tc<128, 128, TST>(a, s);
}

}  // namespace

cudaError_t launch_linear_attn_tc(const LinAttnArgs& a, cudaStream_t s) {
  return a.state == TV_BF16 ? prompt_dims<bf16>(a, s) : prompt_dims<float>(a, s);
}

}  // namespace tv
