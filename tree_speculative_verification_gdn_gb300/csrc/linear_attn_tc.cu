// Linear attention with a decay over prompts on the 5th-generation tensor cores (bf16 I/O).
//
// A prompt (or a segment of one) and head is walked in chunks of C = 128 tokens with the state on
// chip.  With g_i the log2 of the decay from before the chunk to token i, inclusive, and S the
// state before the chunk (dv x dk):
//     P_ij = 2^(g_i - g_j) q_scale q_i.k_j  (j <= i),       O = P V + diag(2^g q_scale) Q S^T,
//     S   <- 2^g_C S + V^T K',                              k'_j = 2^(g_C - g_j) k_j.
// Four products a chunk, all C x 128 x 128.  Q, K and V lie in shared memory as TMA lays them (128-byte
// swizzle); accumulators, the state's transpose, P and K' fill the 512 columns of tensor memory:
//     QK: scores [token i, token j]      A = Q,    B = K
//     QS: O [token i, value]             A = Q,    B = S^T     (bf16 pair); its rows then scaled in place
//     ST: S^T [key column, value]        A = K'^T, B = V       (bf16 pair, tensor memory), added to what bf16
//         leaves of the state; fp32 states: a third part as well (shared memory, in K's place), after QS
//     PV: O, added to                    A = P,    B = V       (bf16 pair, tensor memory, over the scores)
// P, K' and S are fp32 results and enter as value + remainder, two bf16 each (2^-16 left out): one
// bf16 alone would put an error as large as the output's own rounding on every output, and 2^-9 on
// an fp32 state.  For an fp32 state K' has a third part, written over K once the scores have read it:
// without it the state is off by 2.5e-6 of its norm, with it by 5e-7 (32 prompts of 2048 tokens
// 408 -> 476 us; a bf16 state's own rounding is a thousand times either).  The matrix units cut every sum that
// they add to towards zero, a state by 1e-6 and more of itself per thousand tokens; how much depends on
// what is added, so no factor makes up for it (one that did on average was off by 2e-4 after 32768 tokens of
// zero keys).  They add to the state's remainder instead, 2^-9 of it, and its value joins outside
// (batch of 32 prompts 394 -> 405 us).  Exponents only ever go down:
// within 32 x 32 diagonal blocks each 2^(g_i - g_j) is taken directly, elsewhere as
// 2^(g_i - g_r) 2^(g_r - g_j) with r the first row of i's block, so no factor exceeds 1 however fast
// the decay.  g is summed and kept as two floats: after a reset (alpha
// near 0) small differences of large sums remain.
//
// An MMA of this shape reads shared memory at the rate shared memory has (8 KB per 64 clocks), so it,
// not the tensor pipe, is what the products share with TMA and the state's conversion: that is why P
// and K' go through tensor memory (K transposed on the way by ldmatrix) and only S through shared
// memory.
//
// Twenty warps: four turn scores into P (thread = token), four scale and write outputs (thread =
// token), four own the state (thread = key column), four scale the keys; one loads K and Q, one V, one
// issues the MMAs, one sums the decays.  K and Q tiles take turns in a ring of three (K goes back when
// the scores and K' have read it, Q when QS has), V has two; a chunk's outputs leave through its V tile
// by a TMA store (stores of a row by each thread held up every other shared-memory access of the SM).
// (Bringing tiles to L2 a chunk ahead made no difference with this ring.)  One CTA per SM, since five 32 KB tiles and the state's bf16
// pair fill shared memory.  A chunk runs every role's code once, and together it has to stay near the
// instruction cache: hence loops that are not unrolled, and only the first look of a wait inline.
//
// In the pass over states alone (STATE_ONLY: the contributions of a cut prompt's segments) chunks come
// last to first: with the decay from a chunk's end to the segment's folded into K', the state only adds
// up.  Tensor memory holds two K' and two sums: a chunk's starts from zero and joins the segment's in the
// registers of eight warps, 64 values a thread (one prompt of 32768 tokens 310 -> 316 us, a cut fp32 state off
// by 5e-7 instead of up to 6e-6).  The warps without outputs to write make the third part there (the same
// with fp32 states 429 -> 386 us), and one warp loads both K and V, so that two can sum the decays.
//
// Measured on a GB300: 32 prompts of 2048 tokens, 32 heads of 128, 408 us replayed in a graph = 5.4 TB/s, 0.79
// of a plain copy's rate (434 us as a call on changing inputs, 0.74); the tensor pipe is busy half of the
// time, issue slots too.  What bounds it is the chain a chunk hangs on, about 6300 clocks: the state's
// conversion 2600, ST 1300, QS 1500, scaling 600 (P alongside, 3400 from its scores), then PV and, when PV has
// read P, the next scores.  Alone an MMA takes 70 clocks, here about 100, beside the
// other roles' traffic.  Other orders of the four products, more warps on the state (768 threads leave 80
// registers, and K' spills) and copying the state in bulk were slower.
#include <type_traits>

#include "linear_attn.cuh"
#include "tv_async.cuh"
#include "tv_tc.cuh"
#include "tv_tma_host.h"

namespace tv {
namespace {

constexpr int kC = 128;          // tokens per chunk
constexpr int kThreads = 640;    // four roles of four warps; MMA, decay and two TMA warps
constexpr int kHalf = kC * 128;  // bytes of 64 columns of a 128-token tile
constexpr uint32_t kPolls = 1u << 18;
constexpr int kSmemMax = 232448;  // per block
constexpr uint32_t kTransposedA = 1u << 15;  // instruction descriptor: A is MN-major

// TMEM columns; in the pass over states K' of even and odd chunks: from 256 and from 384, their sums from 0 and
// from 128
constexpr uint32_t kColS = 0, kColO = 128, kColQK = 256, kColK = 384;

struct Shared {
  float2 g[2][kC];  // g_i as two floats, by chunk parity
  float f[192];     // 2^(g_r - g_j) of row blocks 1, 2, 3: 32, 64, 96 entries
  uint64_t kq_full[3], kq_empty[3], v_full[2], v_empty[2];
  uint64_t g_full[2], g_empty[2];
  uint64_t qk_done, qs_done, st_done, o_done;           // MMAs complete
  uint64_t s_ready, k_ready, p_ready, o_ready, o_free;  // operands written, outputs read
  uint64_t k_third, st_part;  // fp32 states: third part of K' written, the first two added
  uint64_t o_meet, k_meet;                              // the warps of a role among themselves
  uint64_t drain;
  uint32_t tmem;
  int fail;
};

template <int DK, int DV, bool STATE_ONLY>
struct Plan {
  static constexpr int k = kC * 2 * DK, v = kC * 2 * DV;  // bytes of a tile of K or Q, of V
  static constexpr int nk = 3, nv = 2;                    // tiles in flight
  static constexpr int step = STATE_ONLY ? 1 : 2;         // a chunk's tiles in the ring: K, Q
  static constexpr int at_v = nk * k, at_s = at_v + nv * v;
  static constexpr int s = STATE_ONLY ? 0 : DV * DK * 2;  // the state's bf16 values; as much for its remainders
  static constexpr int bytes = at_s + 2 * s + (int)sizeof(Shared);
  static_assert(bytes <= kSmemMax, "fits an SM");
};

// Place of tile i in a ring of N, and the parity of that place's use.
template <int N>
__device__ __forceinline__ int place(int i) { return i % N; }
template <int N>
__device__ __forceinline__ uint32_t turn(int i) { return (i / N) & 1; }

__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

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
// Waits for the phase of that parity; false once this or another warp has given up.  Executed by a
// whole warp, one answer for all of it.  The first look is inline, the rest is not.
__device__ __noinline__ bool wait_more(Shared& sh, uint64_t* bar, uint32_t parity) {
  bool ok = false;
#pragma unroll 1
  for (uint32_t it = 0; it < kPolls && !ok; ++it) {
    ok = try_wait(bar, parity);
    if (!ok && *reinterpret_cast<volatile int*>(&sh.fail)) break;
  }
  if (!ok) *reinterpret_cast<volatile int*>(&sh.fail) = 1;
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool wait(Shared& sh, uint64_t* bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, try_wait(bar, parity))) return true;
  return wait_more(sh, bar, parity);
}
// The pass over states alone keeps two chunks going: its barriers take turns.
__device__ __forceinline__ uint64_t* state_done(Shared& sh, int n) { return n & 1 ? &sh.qs_done : &sh.st_done; }
__device__ __forceinline__ uint64_t* state_keys(Shared& sh, int n) { return n & 1 ? &sh.p_ready : &sh.k_ready; }
__device__ __forceinline__ uint64_t* state_read(Shared& sh, int n) { return n & 1 ? &sh.o_ready : &sh.s_ready; }
__device__ __forceinline__ uint64_t* state_third(Shared& sh, int n) { return n & 1 ? &sh.st_part : &sh.k_third; }
// Chunk number i of a segment, in the order of the pass: where it starts.
template <bool STATE_ONLY>
__device__ __forceinline__ int chunk_at(const Segment& seg, int i) {
  return seg.t0 + (STATE_ONLY ? (seg.t1 - seg.t0 - 1) / kC - i : i) * kC;
}
__device__ __forceinline__ int chunks_of(const Segment& seg) { return (seg.t1 - seg.t0 + kC - 1) / kC; }

// All 128 threads of a role, by a wait that ends as the others do (a named barrier would wait for ever
// for a warp that gave up).
__device__ __forceinline__ bool meet(Shared& sh, uint64_t* bar, uint32_t& times) {
  mbar_arrive(bar);
  return wait(sh, bar, times++ & 1);
}
// The library's wait, out of line: for the paths after a wait gave up.
__device__ __noinline__ void wait_out(uint64_t* bar, uint32_t parity) { mbar_wait(bar, parity); }

// 32 columns of this thread's lane; tmem_wait_ld() and tmem_join() before their first use.
__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t* r) {
  tmem_ld16_nowait(at, r);
  tmem_ld16_nowait(at + 16, r + 16);
}
template <int N>
__device__ __forceinline__ void tmem_join(uint32_t* r) {
#pragma unroll
  for (int k = 0; k < N; ++k) asm volatile("" : "+r"(r[k]));
}
// 8 and 16 columns, without the wait.
__device__ __forceinline__ void tmem_st8_nowait(uint32_t at, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st16_nowait(uint32_t at, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// 16 lanes x 32 columns: register 4 i + 2 y + x of lane l holds lane 8 x + l / 4, column 8 i + 4 y + l % 4
// -- what transposing 8 x 8 loads of shared memory leave, two 16-bit rows a register.
__device__ __forceinline__ void tmem_st_16x32(uint32_t at, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Four 8 x 8 tiles of 16-bit values, transposed; lane l gives the address of row l % 8 of tile l / 8.
__device__ __forceinline__ void ldsm4t(uint32_t at, uint32_t* v) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(at)
               : "memory");
}

__device__ __forceinline__ float2 pair_of(const uint32_t* s) {
  return make_float2(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float2 rest_of(float2 x, float2 part) { return __ffma2_rn(part, make_float2(-1.f, -1.f), x); }
// What bf16 leaves of x; two columns a word.
__device__ __forceinline__ float2 rest_of(float2 x, uint32_t rounded) {
  return rest_of(x, make_float2(bf16lo(rounded), bf16hi(rounded)));
}
// x as value and remainder; what they leave.
__device__ __forceinline__ float2 split2(float2 x, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(x.x, x.y);
  const float2 rest = rest_of(x, hi);
  lo = pack_bf16x2(rest.x, rest.y);
  return rest_of(rest, lo);
}
// That rest of a key times its decay, instead of the key.
__device__ __forceinline__ uint32_t third_part(uint32_t keys, float scale) {
  uint32_t hi, lo;
  const float2 rest = split2(__fmul2_rn(make_float2(bf16lo(keys), bf16hi(keys)), make_float2(scale, scale)), hi, lo);
  return pack_bf16x2(rest.x, rest.y);
}

// Sums of two floats: hi + lo with |lo| at most half a step of hi.
__device__ __forceinline__ float2 two_sum(float a, float b) {
  const float s = a + b, t = s - a;
  return make_float2(s, (a - (s - t)) + (b - t));
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  const float2 s = two_sum(a.x, b.x);
  const float e = s.y + (a.y + b.y), hi = s.x + e;
  return make_float2(hi, e - (hi - s.x));
}
// 2^g as value and remainder.  A state goes through it once a chunk, often the same one for thousands of
// tokens: a value alone, off by 2^-22, would be off 256 times as far after 32768 tokens.  Below 1/2 little
// is left after a few chunks.
__device__ __forceinline__ float2 decay_of(float2 g) {
  const float x = g.x + g.y;
  if (!(x > -1.f)) return make_float2(ex2_approx(x), 0.f);
  const float less = expm1f(x * 0.69314718f), value = 1.f + less;
  return make_float2(value, less - (value - 1.f));
}
__device__ __forceinline__ float exp2_gap(float2 a, float2 b) { return ex2_approx((a.x - b.x) + (a.y - b.y)); }

// The third part of row r of K' takes the place of K's (pieces in an order without conflicts).
template <int DK>
__device__ __forceinline__ void third_parts(unsigned char* k_tile, int r, float scale) {
#pragma unroll 2
  for (int i = 0; i < DK / 8; ++i) {
    uint4* at = reinterpret_cast<uint4*>(k_tile + i / 8 * kHalf + r * 128 + ((i ^ r) & 7) * 16);
    const uint4 w = *at;
    *at = make_uint4(third_part(w.x, scale), third_part(w.y, scale), third_part(w.z, scale),
                     third_part(w.w, scale));
  }
  fence_proxy_async();
}

template <int DK, int DV, typename TST, bool STATE_ONLY>
__global__ void __launch_bounds__(kThreads, 1)
    linear_attn_tc_kernel(const __grid_constant__ LinAttnArgs a, int units, const __grid_constant__ CUtensorMap mq,
                          const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                          const __grid_constant__ CUtensorMap mo) {
  using L = Plan<DK, DV, STATE_ONLY>;
  constexpr bool THIRD = std::is_same<TST, float>::value;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* s_hi = smem + L::at_s;  // the state's values, then their remainders
  Shared& sh = *reinterpret_cast<Shared*>(s_hi + 2 * L::s);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

  const bool ok = check_seqlens(a);
  if (blockIdx.x == 0 && (STATE_ONLY || a.seg_len == 0))
    for (int b = tid; b < a.B; b += kThreads) a.err[b] = ok ? 0 : TV_ERR_BAD_SEQLEN;
  if (!ok) return;

  if (tid == 0) {
    for (int i = 0; i < 3; ++i) {
      mbar_init(&sh.kq_full[i], 1);
      mbar_init(&sh.kq_empty[i], 1);
      if (i < L::nv) mbar_init(&sh.v_full[i], 1), mbar_init(&sh.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.g_full[i], 1);
      mbar_init(&sh.g_empty[i], !STATE_ONLY ? 16 : THIRD ? 8 : 4);
    }
    mbar_init(&sh.qk_done, 1);
    mbar_init(&sh.qs_done, 1);
    mbar_init(&sh.st_done, 1);
    mbar_init(&sh.o_done, 1);
    mbar_init(&sh.s_ready, STATE_ONLY ? 2 * DV : 128);
    mbar_init(&sh.k_ready, 128);
    mbar_init(&sh.p_ready, 128);
    mbar_init(&sh.o_ready, STATE_ONLY ? 2 * DV : 128);
    mbar_init(&sh.o_free, 128);
    mbar_init(&sh.k_third, 128);
    mbar_init(&sh.st_part, STATE_ONLY ? 128 : 1);
    mbar_init(&sh.o_meet, 128);
    mbar_init(&sh.k_meet, 128);
    mbar_init(&sh.drain, 1);
    sh.fail = 0;
    mbar_fence_init();
  }
  if (warp == 17) tmem_alloc(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t quad = tmem + ((uint32_t)(32 * (warp & 3)) << 16);  // the lanes this warp may touch

  // Every role walks the same units and chunks; n counts chunks over all units.
  int n = 0;
  uint32_t met = 0;  // times the role's warps have met
  bool good = true;
  if (!STATE_ONLY && warp < 4) {
    // ------------------------------------------------ scores to P (thread = token)
    if constexpr (!STATE_ONLY) {
      const uint32_t qk = quad + kColQK;
      float* f = sh.f + (warp == 2 ? 32 : warp == 3 ? 96 : 0);  // 32 * warp entries
#pragma unroll 1
      for (int u = blockIdx.x; u < units && good; u += gridDim.x) {
        const Segment seg = find_segment(a, u);
        if (seg.b < 0) break;
#pragma unroll 1
        for (int t = seg.t0; t < seg.t1; t += kC, ++n) {
          const float2* g = sh.g[n & 1];
          if (!(good = wait(sh, &sh.g_full[n & 1], (n >> 1) & 1))) break;
          const float2 gi = g[tid], gr = g[32 * warp];
          const float ei = exp2_gap(gi, gr) * a.q_scale;
          __syncwarp();  // the last chunk's readers of f are done
#pragma unroll 1
          for (int p = 0; p < warp; ++p) f[lane + 32 * p] = exp2_gap(gr, g[lane + 32 * p]);
          __syncwarp();
          if (!(good = wait(sh, &sh.qk_done, n & 1))) break;
          tc_fence_after();
          // P of tokens 16 p .. + 15 takes the columns of its own scores, values in the first 8, their
          // remainders in the other 8.
          uint32_t s[16];
          tmem_ld16_nowait(qk, s);
#pragma unroll 1
          for (int p = 0; p < 8; ++p) {
            uint32_t hi[8], lo[8];
            const int far = 16 * p - 32 * warp;  // columns of these tokens past the warp's first row
            if (far >= 32) {
#pragma unroll
              for (int c = 0; c < 8; ++c) hi[c] = lo[c] = 0;
            } else {
              tmem_wait_ld();
              tmem_join<16>(s);
              if (far < 0) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                  const float2 x = __fmul2_rn(pair_of(s + 2 * c), *reinterpret_cast<const float2*>(f + 16 * p + 2 * c));
                  split2(__fmul2_rn(x, make_float2(ei, ei)), hi[c], lo[c]);
                }
              } else {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                  const float4 gj = *reinterpret_cast<const float4*>(g + 16 * p + 2 * c);
                  const float e0 = exp2_gap(gi, make_float2(gj.x, gj.y)), e1 = exp2_gap(gi, make_float2(gj.z, gj.w));
                  const float x0 = __uint_as_float(s[2 * c]) * (e0 * a.q_scale);
                  const float x1 = __uint_as_float(s[2 * c + 1]) * (e1 * a.q_scale);
                  split2(make_float2(2 * c <= lane - far ? x0 : 0.f, 2 * c < lane - far ? x1 : 0.f), hi[c], lo[c]);
                }
              }
              if (far < 16) tmem_ld16_nowait(qk + 16 * p + 16, s);
            }
            tmem_st8_nowait(qk + 16 * p, hi);
            tmem_st8_nowait(qk + 16 * p + 8, lo);
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&sh.p_ready);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.g_empty[n & 1]);
        }
      }
    }
  } else if (STATE_ONLY && THIRD && warp >= 4 && warp < 8) {
    // ------------------------------------------------ third part of K' (thread = token)
    const int r = tid - 128;
#pragma unroll 1
    for (int u = blockIdx.x; u < units && good; u += gridDim.x) {
      const Segment seg = find_segment(a, u);
      if (seg.b < 0) break;
      if (seg.index + 1 == seg.count) continue;
      float2 later = make_float2(0.f, 0.f);
      const int chunks = chunks_of(seg);
#pragma unroll 1
      for (int at = 0; at < chunks; ++at, ++n) {
        if (!(good = wait(sh, &sh.g_full[n & 1], (n >> 1) & 1))) break;
        later = add2(later, sh.g[n & 1][kC - 1]);
        const float scale = exp2_gap(later, sh.g[n & 1][r]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.g_empty[n & 1]);
        if (!(good = wait(sh, &sh.kq_full[place<L::nk>(n)], turn<L::nk>(n)))) break;
        if (!(good = wait(sh, state_keys(sh, n), n >> 1 & 1))) break;  // K has been read
        third_parts<DK>(smem + place<L::nk>(n) * L::k, r, scale);
        mbar_arrive(state_third(sh, n));
      }
    }
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------ outputs (thread = token)
    if constexpr (!STATE_ONLY) {
      const uint32_t acc = quad + kColO;
      const int r = tid - 128;
#pragma unroll 1
      for (int u = blockIdx.x; u < units && good; u += gridDim.x) {
        const Segment seg = find_segment(a, u);
        if (seg.b < 0) break;
        bf16* out = static_cast<bf16*>(a.out) + seg.h * DV;
#pragma unroll 1
        for (int t = seg.t0; t < seg.t1; t += kC, ++n) {
          if (!(good = wait(sh, &sh.g_full[n & 1], (n >> 1) & 1))) break;
          const float2 gi = sh.g[n & 1][r];
          const float into = ex2_approx(gi.x + gi.y) * a.q_scale;  // of the state before the chunk
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.g_empty[n & 1]);
          if (!(good = wait(sh, &sh.qs_done, n & 1))) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < DV; c += 32) {
            uint32_t x[32];
            tmem_ld32(acc + c, x);
            tmem_wait_ld();
            tmem_join<32>(x);
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * into);
            tmem_st16_nowait(acc + c, x);
            tmem_st16_nowait(acc + c + 16, x + 16);
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&sh.o_ready);
          if (!(good = wait(sh, &sh.o_done, n & 1))) break;
          tc_fence_after();
          // PV has run, and ST before it: nobody reads this chunk's V tile any more, and it takes the
          // outputs.  A chunk cut short goes out row by row: a whole tile would write into the next
          // prompt's rows.
          const int slot = place<L::nv>(n);
          unsigned char* tile = smem + L::at_v + slot * L::v;
          const bool whole = t + kC <= seg.t1;
          bf16* o = out + (t + r) * a.out_stride;
#pragma unroll 1
          for (int c = 0; c < DV; c += 32) {
            uint32_t x[32];
            tmem_ld32(acc + c, x);
            tmem_wait_ld();
            tmem_join<32>(x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4 w;
              w.x = pack_bf16x2(__uint_as_float(x[8 * i]), __uint_as_float(x[8 * i + 1]));
              w.y = pack_bf16x2(__uint_as_float(x[8 * i + 2]), __uint_as_float(x[8 * i + 3]));
              w.z = pack_bf16x2(__uint_as_float(x[8 * i + 4]), __uint_as_float(x[8 * i + 5]));
              w.w = pack_bf16x2(__uint_as_float(x[8 * i + 6]), __uint_as_float(x[8 * i + 7]));
              if (whole)
                *reinterpret_cast<uint4*>(tile + c / 64 * kHalf + r * 128 + ((c % 64 / 8 + i) ^ (r & 7)) * 16) = w;
              else if (t + r < seg.t1)
                *reinterpret_cast<uint4*>(o + c + 8 * i) = w;
            }
          }
          tc_fence_before();
          mbar_arrive(&sh.o_free);
          if (whole) {
            fence_proxy_async();
            if (!(good = meet(sh, &sh.o_meet, met))) break;
            if (r == 0) {
#pragma unroll
              for (int c = 0; c < DV; c += 64) tma_store_3d(&mo, c, seg.h, t, tile + c / 64 * kHalf);
              bulk_commit();
              bulk_wait_read<0>();
            }
          }
          if (r == 0) mbar_arrive(&sh.v_empty[slot]);
          __syncwarp();
        }
      }
    }
  } else if (STATE_ONLY && ((warp >= 8 && warp < 12) || (DV == 128 && warp < 4))) {
    // ------------------------------------------------ the segments' sums (thread = key column, 64 values)
    // A chunk's sum starts from zero in the matrix units, which cut every sum that they add to, and joins the
    // segment's here.
    if constexpr (STATE_ONLY) {
      const int r = 32 * (warp & 3) + lane, c0 = warp < 4 ? 64 : 0;
      const bool mine = 32 * (warp & 3) < DK;  // warp-uniform
#pragma unroll 1
      for (int u = blockIdx.x; u < units && good; u += gridDim.x) {
        const Segment seg = find_segment(a, u);
        if (seg.b < 0) break;
        if (seg.index + 1 == seg.count) continue;
        float2 sum[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) sum[i] = make_float2(0.f, 0.f);
        const int chunks = chunks_of(seg);
#pragma unroll 1
        for (int at = 0; at < chunks; ++at, ++n) {
          if (!(good = wait(sh, state_done(sh, n), n >> 1 & 1))) break;
          tc_fence_after();
          if (mine) {
#pragma unroll
            for (int c = 0; c < 64; c += 16) {
              uint32_t x[16];
              tmem_ld16_nowait(quad + (n & 1 ? kColO : kColS) + c0 + c, x);
              tmem_wait_ld();
              tmem_join<16>(x);
#pragma unroll
              for (int i = 0; i < 8; ++i) sum[c / 2 + i] = __fadd2_rn(sum[c / 2 + i], pair_of(x + 2 * i));
            }
          }
          tc_fence_before();
          mbar_arrive(state_read(sh, n));
        }
        if (good && mine) {
          float* to = a.slots + ((size_t)u * DV + c0) * DK + r;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            to[2 * i * DK] = sum[i].x;
            to[(2 * i + 1) * DK] = sum[i].y;
          }
        }
      }
    }
  } else if (!STATE_ONLY && warp >= 8 && warp < 12) {
    // ------------------------------------------------ the state (thread = key column)
    const int r = tid - 256;
    const uint32_t row = quad + kColS;
    const bool mine = 32 * (warp - 8) < DK;  // warp-uniform
    // The matrix units cut every sum that they add to towards zero, so they are not given the state: a chunk
    // adds to the decayed remainder of it (2^-9 of the state, what bf16 leaves), and the value, which lies in
    // shared memory for QS, joins it here.  Value and remainder together hold more than a float, so a state
    // that thousands of chunks decay by a little is not rounded by each.
    float kept = 0.f;  // decay of the value in shared memory; 0: none there yet
    float owed = 0.f;  // what rounding has left out of the decays so far, as a fraction
    auto place_of = [&](int c) { return s_hi + c / 64 * (DK * 128) + r * 128 + ((c / 8 % 8) ^ (r & 7)) * 16; };
    // The values of columns c .. c + 15, two a word.
    auto load_values = [&](int c, uint32_t* w) {
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const uint4 x = kept != 0.f ? *reinterpret_cast<const uint4*>(place_of(c + 8 * v)) : make_uint4(0, 0, 0, 0);
        w[4 * v] = x.x, w[4 * v + 1] = x.y, w[4 * v + 2] = x.z, w[4 * v + 3] = x.w;
      }
    };
    auto unpack = [](uint32_t w) { return make_float2(bf16lo(w), bf16hi(w)); };
#pragma unroll 1
    for (int u = blockIdx.x; u < units && good; u += gridDim.x) {
      const Segment seg = find_segment(a, u);
      if (seg.b < 0) break;
      const bool last = seg.index + 1 == seg.count;
      const size_t head = ((size_t)seg.b * a.H + seg.h) * DV * DK + r, slot = (size_t)u * DV * DK + r;
      kept = owed = 0.f;
      if (mine) {
#pragma unroll 1
        for (int c = 0; c < DV; c += 16) {
          float x[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (seg.count > 1) x[i] = a.slots[slot + (c + i) * DK];
            else if (a.S0 != nullptr) x[i] = to_f32(static_cast<const TST*>(a.S0)[head + (c + i) * DK]);
            else x[i] = 0.f;
          }
          tmem_st16_nowait(row + c, reinterpret_cast<const uint32_t*>(x));
        }
        tmem_wait_st();
      }
#pragma unroll 1
      for (int t = seg.t0; t < seg.t1; t += kC, ++n) {
        if (!(good = wait(sh, &sh.g_full[n & 1], (n >> 1) & 1))) break;
        const float2 gc = sh.g[n & 1][kC - 1];
        const float2 decay = decay_of(gc);
        const float more = fmaf(decay.x, owed, decay.y), keep = decay.x + more;
        owed = keep > 0.5f ? __fdividef(more - (keep - decay.x), keep) : 0.f;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.g_empty[n & 1]);
        if (t > seg.t0 && !(good = wait(sh, &sh.st_done, (n - 1) & 1))) break;
        if (n > 0 && !(good = wait(sh, &sh.qs_done, (n - 1) & 1))) break;  // it has read the last S
        tc_fence_after();
        if (mine) {
          uint32_t s[16], w[8];
          tmem_ld16_nowait(row, s);
          load_values(0, w);
          const float2 keep2 = make_float2(keep, keep), kept2 = make_float2(kept, kept), drop2 = make_float2(-kept, -kept);
#pragma unroll 1
          for (int c = 0; c < DV; c += 16) {
            uint32_t x[16], old[8], hi[8], lo[8];
            tmem_wait_ld();
            tmem_join<16>(s);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = s[i];
#pragma unroll
            for (int i = 0; i < 8; ++i) old[i] = w[i];
            if (c + 16 < DV) {
              tmem_ld16_nowait(row + c + 16, s);
              load_values(c + 16, w);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 value = unpack(old[i]), rest = pair_of(x + 2 * i), sum = __ffma2_rn(value, kept2, rest);
              hi[i] = pack_bf16x2(sum.x, sum.y);
              const float2 left = rest_of(rest, __ffma2_rn(value, drop2, unpack(hi[i])));
              lo[i] = pack_bf16x2(left.x, left.y);
              const float2 y = __fmul2_rn(left, keep2);
              x[2 * i] = __float_as_uint(y.x);
              x[2 * i + 1] = __float_as_uint(y.y);
            }
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              unsigned char* to = place_of(c + 8 * v);
              *reinterpret_cast<uint4*>(to) = make_uint4(hi[4 * v], hi[4 * v + 1], hi[4 * v + 2], hi[4 * v + 3]);
              *reinterpret_cast<uint4*>(to + L::s) = make_uint4(lo[4 * v], lo[4 * v + 1], lo[4 * v + 2], lo[4 * v + 3]);
            }
            tmem_st16_nowait(row + c, x);
          }
          tmem_wait_st();
        }
        kept = keep;
        fence_proxy_async();
        tc_fence_before();
        mbar_arrive(&sh.s_ready);
      }
      if (!good) break;
      if (seg.t1 > seg.t0) {
        if (!(good = wait(sh, &sh.st_done, (n - 1) & 1))) break;
        tc_fence_after();
      }
      if (mine && last) {
#pragma unroll 1
        for (int c = 0; c < DV; c += 16) {
          uint32_t s[16];
          tmem_ld16_nowait(row + c, s);
          tmem_wait_ld();
          tmem_join<16>(s);
          uint32_t w[8];
          load_values(c, w);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float value = i % 2 ? bf16hi(w[i / 2]) : bf16lo(w[i / 2]);
            static_cast<TST*>(a.S)[head + (c + i) * DK] = from_f32<TST>(fmaf(value, kept, __uint_as_float(s[i])));
          }
        }
      }
      tc_fence_before();
    }
  } else if (warp >= 12 && warp < 16) {
    // ------------------------------------------------ K', transposed into tensor memory
    // Lane l of a transposing load holds tokens 2 (l % 4) and + 1 of an 8 x 8 tile, key column l / 4.
    // Rows past the segment's end hold another prompt's tokens, or none: K and V rows there become zero.
    const int r = tid - 384;
    const uint32_t keys = quad + kColK;
    const bool mine = 32 * (warp - 12) < DK;  // warp-uniform
#pragma unroll 1
    for (int u = blockIdx.x; u < units && good; u += gridDim.x) {
      const Segment seg = find_segment(a, u);
      if (seg.b < 0) break;
      if (STATE_ONLY && seg.index + 1 == seg.count) continue;
      float2 later = make_float2(0.f, 0.f);  // log2 of the decay from the chunk's end to the segment's
      const int chunks = chunks_of(seg);
#pragma unroll 1
      for (int at = 0; at < chunks; ++at, ++n) {
        const int t = chunk_at<STATE_ONLY>(seg, at);
        const int rows = seg.t1 - t;
        const int ik = n * L::step;
        unsigned char* k_tile = smem + place<L::nk>(ik) * L::k;
        const float2* g = sh.g[n & 1];
        if (!(good = wait(sh, &sh.g_full[n & 1], (n >> 1) & 1))) break;
        if (!(good = wait(sh, &sh.kq_full[place<L::nk>(ik)], turn<L::nk>(ik)))) break;
        // the update has read the last K' of this place
        if (STATE_ONLY ? n > 1 && !(good = wait(sh, state_done(sh, n), (n - 2) >> 1 & 1))
                       : n > 0 && !(good = wait(sh, THIRD ? &sh.st_part : &sh.st_done, (n - 1) & 1)))
          break;
        tc_fence_after();
        if (rows < kC) {
          if (!(good = wait(sh, &sh.v_full[place<L::nv>(n)], turn<L::nv>(n)))) break;
          auto clear = [&](unsigned char* tile, int columns) {  // eight 16-byte pieces a row and 64 columns
#pragma unroll 1
            for (int half = 0; half < columns / 64; ++half)
#pragma unroll 1
              for (int i = rows * 8 + r; i < kC * 8; i += 128)
                reinterpret_cast<uint4*>(tile + half * kHalf)[i] = make_uint4(0, 0, 0, 0);
          };
          clear(k_tile, DK);
          clear(smem + L::at_v + place<L::nv>(n) * L::v, DV);
          fence_proxy_async();
          if (!(good = meet(sh, &sh.k_meet, met))) break;
        }
        float2 gc = g[kC - 1];
        if (STATE_ONLY) gc = later = add2(later, gc);
        if (mine) {
#pragma unroll 1
          for (int part = 0; part < 2; ++part) {  // 64 tokens
            float2 scale[8];                      // of tokens 8 i + 2 (lane % 4) and + 1
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 gj = *reinterpret_cast<const float4*>(g + 64 * part + 8 * i + 2 * (lane & 3));
              scale[i] = make_float2(exp2_gap(gc, make_float2(gj.x, gj.y)), exp2_gap(gc, make_float2(gj.z, gj.w)));
            }
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {  // 16 key columns
              const int c = 32 * (warp - 12) + 16 * half + (lane & 8), j0 = (lane & 7) + (lane & 16) / 2;
              const uint32_t from = smem_addr(k_tile) + c / 64 * kHalf + (64 * part + j0) * 128 +
                                    (((c % 64 / 8) ^ (j0 & 7)) << 4);
              uint32_t hi[16], lo[16];
#pragma unroll
              for (int i = 0; i < 4; ++i) {  // 16 tokens
                uint32_t w[4];
                ldsm4t(from + 16 * i * 128, w);
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  split2(__fmul2_rn(make_float2(bf16lo(w[x]), bf16hi(w[x])), scale[2 * i + x / 2]), hi[4 * i + x],
                         lo[4 * i + x]);
              }
              const uint32_t to = keys - (STATE_ONLY && !(n & 1) ? 128 : 0) + ((uint32_t)(16 * half) << 16) + 32 * part;
              tmem_st_16x32(to, hi);
              tmem_st_16x32(to + 64, lo);
            }
          }
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(STATE_ONLY ? state_keys(sh, n) : &sh.k_ready);
        if (THIRD && !STATE_ONLY) {
          if (!(good = wait(sh, &sh.k_ready, n & 1))) break;  // all have read the keys,
          if (!(good = wait(sh, &sh.qk_done, n & 1))) break;  // and the scores too
          third_parts<DK>(k_tile, r, exp2_gap(gc, g[r]));
          mbar_arrive(&sh.k_third);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.g_empty[n & 1]);
      }
      if (STATE_ONLY && r == 0) a.decay[u] = decay_of(later);
    }
  } else if (warp == 19 || (!STATE_ONLY && warp == 16)) {
    // ------------------------------------------------ TMA loads
    auto load = [&](const CUtensorMap* map, unsigned char* to, int columns, int h, int t, uint64_t* full) {
      if (lane == 0) {
        mbar_arrive_expect_tx(full, columns / 64 * kHalf);
        tma_load_3d(to, map, 0, h, t, full);
        if (columns > 64) tma_load_3d(to + kHalf, map, 64, h, t, full);
      }
      __syncwarp();
    };
    // One warp K and Q, one V; in the pass over states one both.
    const bool keys = warp == 19, values = STATE_ONLY || !keys;
    int nk = 0, nv = 0;  // tiles asked for
#pragma unroll 1
    for (int u = blockIdx.x; u < units && good; u += gridDim.x) {
      const Segment seg = find_segment(a, u);
      if (seg.b < 0) break;
      if (STATE_ONLY && seg.index + 1 == seg.count) continue;
      const int h = seg.h, hk = h / (a.H / a.Hk);
      const int chunks = chunks_of(seg);
      int tile = 0;  // of the segment's K and Q tiles, the next
#pragma unroll 1
      for (int at = 0; at < chunks && good; ++at) {
        if (keys) {
          // K's place is free before V's: a chunk ahead where one warp loads both
          const int to = L::step * min(at + (STATE_ONLY ? 2 : 1), chunks);
#pragma unroll 1
          for (; tile < to; ++tile, ++nk) {
            const int i = place<L::nk>(nk);
            if (nk >= L::nk && !(good = wait(sh, &sh.kq_empty[i], turn<L::nk>(nk) ^ 1))) break;
            load(tile % L::step == 0 ? &mk : &mq, smem + i * L::k, DK, hk, chunk_at<STATE_ONLY>(seg, tile / L::step),
                 &sh.kq_full[i]);
          }
        }
        if (values && good) {
          const int i = place<L::nv>(nv);
          if (nv >= L::nv && !(good = wait(sh, &sh.v_empty[i], turn<L::nv>(nv) ^ 1))) break;
          load(&mv, smem + L::at_v + i * L::v, DV, h, chunk_at<STATE_ONLY>(seg, at), &sh.v_full[i]);
          ++nv;
        }
      }
    }
    if (!good) {  // leave no copy in flight behind: the last ones
#pragma unroll 1
      for (int i = 1; i <= L::nk && i <= nk; ++i) wait_out(&sh.kq_full[place<L::nk>(nk - i)], turn<L::nk>(nk - i));
#pragma unroll 1
      for (int i = 1; i <= L::nv && i <= nv; ++i) wait_out(&sh.v_full[place<L::nv>(nv - i)], turn<L::nv>(nv - i));
    }
  } else if (warp == 17) {
    // ------------------------------------------------ MMAs
    // The next unit that has tokens, from u on; its number, and its chunks in `chunks`.
    auto find = [&](int u, int& chunks) {
#pragma unroll 1
      for (; u < units; u += gridDim.x) {
        const Segment seg = find_segment(a, u);
        if (seg.b < 0) break;
        chunks = (seg.t1 - seg.t0 + kC - 1) / kC;
        if (chunks > 0 && !(STATE_ONLY && seg.index + 1 == seg.count)) return u;
      }
      chunks = 0;
      return units;
    };
    const uint32_t base = smem_addr(smem), st = smem_addr(s_hi);
    // Descriptors count 16 bytes; only their start differs, so the others are these plus an offset.
    const uint64_t by_rows = sw128_desc(0), by_columns = sw128_mn_desc(0, kHalf), state = sw128_mn_desc(st, DK * 128);
    auto start = [&](int offset) { return __shfl_sync(0xffffffffu, (base + offset) >> 4, 0); };
    // Scores of chunk n, whose tiles have landed.
    auto landed = [&](int n) {
      const int i = n * L::step;
      return wait(sh, &sh.kq_full[place<L::nk>(i)], turn<L::nk>(i)) &&
             wait(sh, &sh.kq_full[place<L::nk>(i + 1)], turn<L::nk>(i + 1));
    };
    auto scores = [&](uint64_t dq, uint64_t dk) {
      constexpr uint32_t id = idesc_bf16_f32(kC, kC);
#pragma unroll
      for (int c = 0; c < DK; c += 16) {
        const int off = (c / 64 * kHalf + c % 64 * 2) >> 4;
        mma_bf16(tmem + kColQK, dq + off, dk + off, id, c > 0);
      }
      mma_commit(&sh.qk_done);
    };
    auto q_rows = [&](int n) { return by_rows + start(place<L::nk>(n * L::step + 1) * L::k); };
    auto k_rows = [&](int n) { return by_rows + start(place<L::nk>(n * L::step) * L::k); };
    int chunks, later;
    int u = find(blockIdx.x, chunks);
    if (!STATE_ONLY && u < units && (good = landed(0))) {
      tc_fence_after();
      const uint64_t dq = q_rows(0), dk = k_rows(0);
      if (elect_one()) scores(dq, dk);
      __syncwarp();
    }
#pragma unroll 1
    while (u < units && good) {
      const int next = find(u + gridDim.x, later);
#pragma unroll 1
      for (int i = 0; i < chunks; ++i, ++n) {
        const int iv = place<L::nv>(n);
        if (STATE_ONLY) {
          if (n > 1 && !(good = wait(sh, state_read(sh, n), (n - 2) >> 1 & 1))) break;
          if (!(good = wait(sh, state_keys(sh, n), n >> 1 & 1))) break;
        } else {
          if (!(good = wait(sh, &sh.s_ready, n & 1))) break;
          if (!(good = wait(sh, &sh.k_ready, n & 1))) break;
        }
        if (!(good = wait(sh, &sh.v_full[iv], turn<L::nv>(n)))) break;
        tc_fence_after();
        // ST first, so that the next K' is made while QS and PV run.
        // M = 128 key columns; with dk = 64 the upper 64 are whatever those lanes hold, and nobody reads
        // them.
        constexpr uint32_t idv = idesc_bf16_f32(kC, DV, true);
        const uint64_t dv = by_columns + start(L::at_v + iv * L::v);
        const uint64_t rest = by_columns + start(place<L::nk>(n * L::step) * L::k);
        const uint32_t to = tmem + (STATE_ONLY && n & 1 ? kColO : kColS);
        auto add_third = [&] {
#pragma unroll
          for (int c = 0; c < kC; c += 16) mma_bf16(to, rest + c * 8, dv + c * 8, idv | kTransposedA, 1);
        };
        if (elect_one()) {
          if (!THIRD) mma_commit(&sh.kq_empty[place<L::nk>(n * L::step)]);  // the scores have read K, and K' is made
#pragma unroll 1
          for (int part = 1; part >= 0; --part)  // remainders first: their sum is small, and cut by little
#pragma unroll
            for (int c = 0; c < kC; c += 16)
              mma_bf16_tmem_a(to, tmem + kColK - (STATE_ONLY && !(n & 1) ? 128 : 0) + 64 * part + c / 2,
                              dv + c * 8, idv, !STATE_ONLY || (1 - part) + c > 0);
          if (!STATE_ONLY) mma_commit(THIRD ? &sh.st_part : &sh.st_done);
        }
        __syncwarp();
        if (STATE_ONLY) {
          if (THIRD && !(good = wait(sh, state_third(sh, n), n >> 1 & 1))) break;
          if (elect_one()) {
            if (THIRD) {
              add_third();
              mma_commit(&sh.kq_empty[place<L::nk>(n * L::step)]);
            }
            mma_commit(state_done(sh, n));
            mma_commit(&sh.v_empty[iv]);
          }
          __syncwarp();
          continue;
        }
        if (n > 0 && !(good = wait(sh, &sh.o_free, (n - 1) & 1))) break;
        tc_fence_after();
        constexpr uint32_t ids = idesc_bf16_f32(kC, DV, true);
        const uint64_t this_q = q_rows(n);
        if (elect_one()) {
#pragma unroll 1
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int c = 0; c < DK; c += 16)
              mma_bf16(tmem + kColO, this_q + ((c / 64 * kHalf + c % 64 * 2) >> 4), state + ((part * L::s + c * 128) >> 4),
                       ids, part + c > 0);
          mma_commit(&sh.qs_done);
          mma_commit(&sh.kq_empty[place<L::nk>(n * L::step + 1)]);
        }
        __syncwarp();
        if (THIRD) {
          if (!(good = wait(sh, &sh.k_third, n & 1))) break;
          if (elect_one()) {
            add_third();
            mma_commit(&sh.st_done);
            mma_commit(&sh.kq_empty[place<L::nk>(n * L::step)]);
          }
          __syncwarp();
        }
        const bool more = i + 1 < chunks || next < units;
        if (!(good = wait(sh, &sh.p_ready, n & 1))) break;
        if (!(good = wait(sh, &sh.o_ready, n & 1))) break;
        tc_fence_after();
        const uint64_t next_q = q_rows(n + 1), next_k = k_rows(n + 1);
        if (elect_one()) {
#pragma unroll 1
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int c = 0; c < kC; c += 16)
              mma_bf16_tmem_a(tmem + kColO, tmem + kColQK + c + 8 * part, dv + c * 8, idv, 1);
          mma_commit(&sh.o_done);
        }
        __syncwarp();
        if (more) {
          if (!(good = landed(n + 1))) break;
          // The scores go over P, which PV reads: MMAs are kept in order on one accumulator, and these have two.
          if (!(good = wait(sh, &sh.o_done, n & 1))) break;
          tc_fence_after();
          if (elect_one()) scores(next_q, next_k);
          __syncwarp();
        }
      }
      u = next;
      chunks = later;
    }
  } else if (warp == 18 || (STATE_ONLY && warp == 16)) {
    // ------------------------------------------------ decays: four tokens a lane
    // In the pass over states, whose other steps are short, two warps take turns.
    constexpr int kTurns = STATE_ONLY ? 2 : 1;
    const int turn = warp == 16;
#pragma unroll 1
    for (int u = blockIdx.x; u < units && good; u += gridDim.x) {
      const Segment seg = find_segment(a, u);
      if (seg.b < 0) break;
      if (STATE_ONLY && seg.index + 1 == seg.count) continue;
      const float* al = a.alpha + seg.h;
      float next[4];  // the next chunk's decays, on their way
      auto fetch = [&](int t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = t + 4 * lane + i;  // past the prompt's end nothing decays
          next[i] = tok < seg.t1 ? __ldg(al + tok * a.alpha_stride) : 1.f;
        }
      };
      const int chunks = chunks_of(seg);
      const int first = (n ^ turn) & (kTurns - 1), past = n + chunks;
      n += first;
      if (first < chunks) fetch(chunk_at<STATE_ONLY>(seg, first));
#pragma unroll 1
      for (int at = first; at < chunks; at += kTurns, n += kTurns) {
        float2 sum[4];
        // alpha = 0 forgets everything: 2^-1000 times any state is 0 in fp32
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = make_float2(next[i] == 0.f ? -1000.f : log2f(next[i]), 0.f);
        if (at + kTurns < chunks) fetch(chunk_at<STATE_ONLY>(seg, at + kTurns));
#pragma unroll
        for (int i = 1; i < 4; ++i) sum[i] = add2(sum[i - 1], sum[i]);
        float2 up = sum[3];
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
          const float2 below = make_float2(__shfl_up_sync(0xffffffffu, up.x, o), __shfl_up_sync(0xffffffffu, up.y, o));
          if (lane >= o) up = add2(below, up);
        }
        up = make_float2(__shfl_up_sync(0xffffffffu, up.x, 1), __shfl_up_sync(0xffffffffu, up.y, 1));
        if (n >= 2 && !(good = wait(sh, &sh.g_empty[n & 1], ((n >> 1) - 1) & 1))) break;
        float4* g = reinterpret_cast<float4*>(sh.g[n & 1] + 4 * lane);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (lane > 0) sum[i] = add2(up, sum[i]);
        g[0] = make_float4(sum[0].x, sum[0].y, sum[1].x, sum[1].y);
        g[1] = make_float4(sum[2].x, sum[2].y, sum[3].x, sum[3].y);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.g_full[n & 1]);
      }
      n = past;
    }
  }
  __syncwarp();
  // Every MMA has completed: the state's and the outputs' warps waited for their last.  After a wait
  // that gave up the last ones issued may still run, so wait for them too.
  if (warp == 17 && *reinterpret_cast<volatile int*>(&sh.fail)) {
    if (lane == 0) mma_commit(&sh.drain);
    __syncwarp();
    wait_out(&sh.drain, 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 17) tmem_dealloc(tmem, 512);
  if (sh.fail && warp == 0)
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
      const Segment seg = find_segment(a, u);
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
  fn<<<units < sms ? units : sms, kThreads, L::bytes, s>>>(a, units, m[0], m[1], m[2], m[3]);
  return cudaGetLastError();
}

template <int DK, int DV, typename TST>
cudaError_t prompt_tc(const LinAttnArgs& a, cudaStream_t s) {
  CUtensorMap m[4];
  if (!token_map(&m[0], a.q, DK, a.Hk, a.T, a.q_stride) || !token_map(&m[1], a.k, DK, a.Hk, a.T, a.k_stride) ||
      !token_map(&m[2], a.v, DV, a.H, a.T, a.v_stride) || !token_map(&m[3], a.out, DV, a.H, a.T, a.out_stride))
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
