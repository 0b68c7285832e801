// Linear attention with a decay per head: S_t = alpha_t S_{t-1} + v_t k_t^T, o_t = S_t (q_scale q_t).
//
//   linear_attn_kernel       whole prompts, token by token, on the CUDA cores: fp32 I/O, and bf16 prompts
//                            that are too short for chunks of 128 tokens
//   linear_attn_scan_kernel  the states that the segments of a cut prompt start from
//   linear_attn_step_kernel  one token of every sequence
//
// Row r of S needs k_t, q_t, alpha_t and v_t[r] only, so rows are independent: a CTA of the prompt
// kernel keeps kRows rows in registers, eight lanes a row and four rows a lane, and walks the tokens.
// It is bound by the multiply-adds, three a state element and token, and by the loads of k and q from
// shared memory that feed them: four rows a lane share each load, columns go in pairs (32 prompts of
// 300 fp32 tokens, 32 heads: one row a lane 1418 us, two 866, four 702, four in pairs 627).
// fp32 prompts may be long.  A state that takes in every decay as it comes is rounded by each, the same way for
// thousands of tokens where decays are near to 1: 2e-4 of itself after 32768.  There, with D_t the decay since the
// state was last scaled,
//     Z_t = Z_{t-1} + (v_t / D_t) k_t^T,     o_t = D_t q_scale Z_t q_t:
// two multiply-adds and one rounding a token (the 627 us above become 571).  Z is scaled by D, a product of two floats, only once that is below a
// half.  kBlock tokens that decay below 2^-20 together (1 / D leaves the range) are walked as they stand, like bf16
// prompts, which come here only when they are short.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "linear_attn.cuh"

namespace tv {
namespace {

// ------------------------------------------------------------------ prompts, token by token
constexpr int kThreads = 128;
constexpr int kLPR = 8;                                // lanes per state row
constexpr int kRPL = 4;                                // rows per lane
constexpr int kRows = kThreads / kLPR * kRPL;          // rows per CTA
constexpr int kBlock = 16;                             // tokens staged at a time
constexpr float kDirect = 1.f / (1 << 20);             // decay of a block below which it is walked as it stands

// Eight elements as stored, then as floats.
template <typename T> struct Raw8;
template <> struct Raw8<bf16> {
  uint4 w;
  __device__ __forceinline__ void load(const bf16* p) { w = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float* o) const { unpack8(w, o); }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float* o) const {
    o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
    o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
  }
};

// Sums v[0..7] over eight consecutive lanes; lane l of the eight receives the total of v[l].
// Halving the values with every exchange takes 7 shuffles where eight sums one by one take 24.
__device__ __forceinline__ float sum8(const float* v, int l) {
  float x[4], y[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float mine = (l & 4) ? v[i + 4] : v[i], give = (l & 4) ? v[i] : v[i + 4];
    x[i] = mine + __shfl_xor_sync(0xffffffffu, give, 4);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float mine = (l & 2) ? x[i + 2] : x[i], give = (l & 2) ? x[i] : x[i + 2];
    y[i] = mine + __shfl_xor_sync(0xffffffffu, give, 2);
  }
  const float mine = (l & 1) ? y[1] : y[0], give = (l & 1) ? y[0] : y[1];
  return mine + __shfl_xor_sync(0xffffffffu, give, 1);
}

// Product of two numbers of two floats each, the second at most half a step of the first.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  const float x = a.x * b.x, y = fmaf(a.x, b.x, -x) + fmaf(a.x, b.y, a.y * b.x), hi = x + y;
  return make_float2(hi, y - (hi - x));
}

// One segment of one prompt, kRows rows of one head's state.  STATE_ONLY: the segment's own
// contribution to the state (from zero) and its total decay, into the workspace.
template <typename TIO, typename TST, int DK, int DV, bool STATE_ONLY>
__global__ void __launch_bounds__(kThreads) linear_attn_kernel(LinAttnArgs a) {
  constexpr bool SPLIT = std::is_same<TIO, float>::value;  // S = D Z
  constexpr int CPL = DK / kLPR;         // columns per lane: four at 4 l + 32 j
  constexpr int kSlabs = DV / kRows;
  constexpr int kVec = kBlock * DK / 8 / kThreads;   // 8-column vectors of k (and of q) per thread
  constexpr int kVPT = kBlock * kRows / kThreads;    // values of v per thread
  __shared__ __align__(16) float s_k[kBlock][DK], s_q[STATE_ONLY ? 1 : kBlock][DK], s_v[kBlock][kRows];
  __shared__ __align__(16) float s_o[STATE_ONLY ? 1 : kBlock][kRows];
  __shared__ float s_a[kBlock];

  const int tid = threadIdx.x;
  const int slab = blockIdx.x % kSlabs, u = blockIdx.x / kSlabs;
  const bool ok = check_seqlens(a);
  if (blockIdx.x == 0 && (STATE_ONLY || a.seg_len == 0))
    for (int b = tid; b < a.B; b += kThreads) a.err[b] = ok ? 0 : TV_ERR_BAD_SEQLEN;
  if (!ok) return;
  const Segment seg = find_segment(a, u);
  if (seg.b < 0 || (STATE_ONLY && seg.index + 1 == seg.count)) return;

  const int h = seg.h, hk = h / (a.H / a.Hk);
  const TIO* kp = static_cast<const TIO*>(a.k) + hk * DK;
  const TIO* qp = static_cast<const TIO*>(a.q) + hk * DK;
  const TIO* vp = static_cast<const TIO*>(a.v) + h * DV + slab * kRows;
  TIO* op = static_cast<TIO*>(a.out) + h * DV + slab * kRows;

  const int l = tid % kLPR, row0 = tid / kLPR * kRPL;  // this lane's first row of the slab
  float2 s2[kRPL][CPL / 2];  // column pairs of S, or of Z
  float(&s)[kRPL][CPL] = reinterpret_cast<float(&)[kRPL][CPL]>(s2);
  const size_t head = (size_t)seg.b * a.H + h, slot = u;
#pragma unroll
  for (int r = 0; r < kRPL; ++r) {
    const int at = (slab * kRows + row0 + r) * DK + 4 * l;
#pragma unroll
    for (int j = 0; j < CPL / 4; ++j) {
      if (!STATE_ONLY && seg.count > 1) {
        load_vec_rw<4>(a.slots + slot * DV * DK + at + 32 * j, s[r] + 4 * j);
      } else if (!STATE_ONLY && a.S0 != nullptr) {
        load_vec_rw<4>(static_cast<const TST*>(a.S0) + head * DV * DK + at + 32 * j, s[r] + 4 * j);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) s[r][4 * j + c] = 0.f;
      }
    }
  }
  float2 since = make_float2(1.f, 0.f), total = since;  // D, and the segment's decay so far
  auto scale = [&] {  // Z becomes S
#pragma unroll
    for (int r = 0; r < kRPL; ++r)
#pragma unroll
      for (int c = 0; c < CPL / 2; ++c)
        s2[r][c] = __ffma2_rn(s2[r][c], make_float2(since.x, since.x),
                              __fmul2_rn(s2[r][c], make_float2(since.y, since.y)));
    since = make_float2(1.f, 0.f);
  };

  Raw8<TIO> rk[kVec], rq[kVec];
  TIO rv[kVPT];
  float ra = 1.f;
  // Tokens past the segment's end enter as k = q = v = 0 and alpha = 1: they leave the state alone.
  auto fetch = [&](int t) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int e = tid + i * kThreads, tok = t + e / (DK / 8), c = e % (DK / 8) * 8;
      if (tok < seg.t1) {
        rk[i].load(kp + tok * a.k_stride + c);
        if (!STATE_ONLY) rq[i].load(qp + tok * a.q_stride + c);
      } else {
        rk[i].zero();
        rq[i].zero();
      }
    }
#pragma unroll
    for (int i = 0; i < kVPT; ++i) {
      const int e = tid + i * kThreads, tok = t + e / kRows;
      rv[i] = tok < seg.t1 ? vp[tok * a.v_stride + e % kRows] : from_f32<TIO>(0.f);
    }
    const int tok = t + tid % kBlock;  // every warp has them all
    ra = tok < seg.t1 ? __ldg(a.alpha + tok * a.alpha_stride + h) : 1.f;
  };
  fetch(seg.t0);
  auto last_of = [](float2 x) {
    return make_float2(__shfl_sync(0xffffffffu, x.x, kBlock - 1), __shfl_sync(0xffffffffu, x.y, kBlock - 1));
  };
  for (int t = seg.t0; t < seg.t1; t += kBlock) {
    float2 now = make_float2(1.f, 0.f);  // SPLIT: D_i in lane i % kBlock, and 1 / D_i
    float inverse = 1.f;
    bool direct = true;
    if (SPLIT) {
      float2 p = make_float2(ra, 0.f);  // the product of the block's decays up to token i
#pragma unroll
      for (int o = 1; o < kBlock; o <<= 1) {
        const float2 up = make_float2(__shfl_up_sync(0xffffffffu, p.x, o, kBlock),
                                      __shfl_up_sync(0xffffffffu, p.y, o, kBlock));
        const float2 both = mul2(up, p);
        if (tid % kBlock >= o) p = both;
      }
      const float2 whole = last_of(p);
      direct = !(whole.x >= kDirect);
      if (direct) {
        scale();
      } else {
        now = mul2(since, p);
        inverse = 1.f / now.x;
      }
      if (STATE_ONLY) total = mul2(total, whole);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int e = tid + i * kThreads, tok = e / (DK / 8), c = e % (DK / 8) * 8;
      float x[8];
      rk[i].get(x);
      store_vec<8>(&s_k[tok][c], x);
      if (!STATE_ONLY) {
        rq[i].get(x);
        store_vec<8>(&s_q[tok][c], x);
      }
    }
#pragma unroll
    for (int i = 0; i < kVPT; ++i) {
      const int e = tid + i * kThreads;  // one token a warp
      s_v[e / kRows][e % kRows] = to_f32(rv[i]) * (SPLIT ? __shfl_sync(0xffffffffu, inverse, e / kRows) : 1.f);
    }
    if (tid < kBlock) s_a[tid] = ra;
    __syncthreads();
    if (t + kBlock < seg.t1) fetch(t + kBlock);
    // Eight tokens; with SOME only those of the segment.
    auto walk = [&](int u, auto some, auto as_it_stands) {
      constexpr bool SOME = decltype(some)::value, DIRECT = decltype(as_it_stands)::value;
      float dot[kRPL][8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int r = 0; r < kRPL; ++r) dot[r][i] = 0.f;
        if (SOME && t + u + i >= seg.t1) continue;  // the same for the whole CTA
        const float al = DIRECT ? s_a[u + i] : 1.f;
        float2 v[kRPL], sum[kRPL];
#pragma unroll
        for (int r = 0; r < kRPL; ++r) {
          const float x = s_v[u + i][row0 + r];
          v[r] = make_float2(x, x);
          sum[r] = make_float2(0.f, 0.f);
        }
        const float2 al2 = make_float2(al, al);
#pragma unroll
        for (int j = 0; j < CPL / 4; ++j) {
          const float4 k4 = *reinterpret_cast<const float4*>(&s_k[u + i][4 * l + 32 * j]);
          const float2 kk[2] = {make_float2(k4.x, k4.y), make_float2(k4.z, k4.w)};
          float4 q4 = make_float4(0, 0, 0, 0);
          if (!STATE_ONLY) q4 = *reinterpret_cast<const float4*>(&s_q[u + i][4 * l + 32 * j]);
          const float2 qq[2] = {make_float2(q4.x, q4.y), make_float2(q4.z, q4.w)};
#pragma unroll
          for (int r = 0; r < kRPL; ++r)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float2& x = s2[r][2 * j + c];
              x = __ffma2_rn(v[r], kk[c], DIRECT ? __fmul2_rn(al2, x) : x);
              if (!STATE_ONLY) sum[r] = __ffma2_rn(x, qq[c], sum[r]);
            }
        }
#pragma unroll
        for (int r = 0; r < kRPL; ++r) dot[r][i] = sum[r].x + sum[r].y;
      }
      if (!STATE_ONLY) {
        const float by = SPLIT ? __shfl_sync(0xffffffffu, now.x, u + l) * a.q_scale : a.q_scale;
#pragma unroll
        for (int r = 0; r < kRPL; ++r) s_o[u + l][row0 + r] = sum8(dot[r], l) * by;
      }
    };
    const std::true_type yes;
    const std::false_type no;
#pragma unroll 1
    for (int u = 0; u < kBlock && t + u < seg.t1; u += 8) {
      const bool whole = t + u + 8 <= seg.t1;
      if constexpr (SPLIT) {
        if (!direct) {
          if (whole) walk(u, no, no);
          else walk(u, yes, no);
          continue;
        }
      }
      if (whole) walk(u, no, yes);
      else walk(u, yes, yes);
    }
    if (SPLIT && !direct) {
      since = last_of(now);
      if (!(since.x >= 0.5f)) scale();
    }
    if (!STATE_ONLY) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kVPT / 4; ++i) {
        const int e = (tid + i * kThreads) * 4, tok = t + e / kRows;
        if (tok < seg.t1) store_vec<4>(op + tok * a.out_stride + e % kRows, &s_o[e / kRows][e % kRows]);
      }
    }
  }
  const bool last = seg.index + 1 == seg.count;
  if (!STATE_ONLY && !last) return;
  if (SPLIT) scale();
#pragma unroll
  for (int r = 0; r < kRPL; ++r) {
    const int at = (slab * kRows + row0 + r) * DK + 4 * l;
#pragma unroll
    for (int j = 0; j < CPL / 4; ++j) {
      if (STATE_ONLY) store_vec<4>(a.slots + slot * DV * DK + at + 32 * j, s[r] + 4 * j);
      else store_vec<4>(static_cast<TST*>(a.S) + head * DV * DK + at + 32 * j, s[r] + 4 * j);
    }
  }
  if (STATE_ONLY && slab == 0 && tid == 0) a.decay[slot] = total;
}

// ------------------------------------------------------------------ states between segments
// Slot s of a cut prompt holds the segment's own contribution dS_s and receives the state that
// segment s starts from: X_0 = S0, X_{s+1} = decay_s X_s + dS_s, by two floats (a decay near 1 would round an
// element the same way in every segment).  Four columns a thread.  S0 itself
// is copied into slot 0, so that the last segment may write S over it while the first one runs.
template <typename TST>
__global__ void __launch_bounds__(256) linear_attn_scan_kernel(LinAttnArgs a, int parts) {
  if (!check_seqlens(a)) return;
  const int part = blockIdx.x % parts, h = blockIdx.x / parts % a.H, b = blockIdx.x / parts / a.H;
  const int n = segments_of(__ldg(a.cu + b + 1) - __ldg(a.cu + b), a.seg_len);
  if (n == 1) return;
  const int first = first_segment(a, b);
  const size_t size = (size_t)a.dv * a.dk, at = ((size_t)part * 256 + threadIdx.x) * 4;
  if (at >= size) return;
  float x[4] = {0.f, 0.f, 0.f, 0.f}, rest[4] = {0.f, 0.f, 0.f, 0.f};  // X as two floats
  if (a.S0 != nullptr) load_vec_rw<4>(static_cast<const TST*>(a.S0) + ((size_t)b * a.H + h) * size + at, x);
  // Four segments' values are asked for before the first is needed (one by one, a segment took 4 us).
  constexpr int kAhead = 4;
  const size_t stride = (size_t)a.H * size;
  float* p = a.slots + ((size_t)first * a.H + h) * size + at;
  const float2* f = a.decay + (size_t)first * a.H + h;
  for (int s = 0; s < n; s += kAhead, p += kAhead * stride, f += kAhead * a.H) {
    float d[kAhead][4];
    float2 g[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (s + i + 1 < n) {
        load_vec_rw<4>(p + i * stride, d[i]);
        g[i] = f[i * a.H];
      }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (s + i < n) {
        store_vec<4>(p + i * stride, x);
        if (s + i + 1 < n)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float2 kept = mul2(g[i], make_float2(x[c], rest[c]));
            const float sum = kept.x + d[i][c], part = sum - kept.x;
            const float low = kept.y + ((kept.x - (sum - part)) + (d[i][c] - part));
            x[c] = sum + low;
            rest[c] = low - (x[c] - sum);
          }
      }
  }
}

template <typename TIO, typename TST, int DK, int DV>
cudaError_t prompt_simt(const LinAttnArgs& a, cudaStream_t s) {
  const long long segments = a.seg_len > 0 ? (long long)a.B + a.T / a.seg_len : a.B;
  const long long grid = segments * a.H * (DV / kRows);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if constexpr (std::is_same<TIO, float>::value) {  // bf16 prompts are cut by the tensor-core form alone
    if (a.seg_len > 0) {
      linear_attn_kernel<TIO, TST, DK, DV, true><<<(unsigned)grid, kThreads, 0, s>>>(a);
      const cudaError_t e = launch_linear_attn_scan(a, s);
      if (e != cudaSuccess) return e;
    }
  }
  linear_attn_kernel<TIO, TST, DK, DV, false><<<(unsigned)grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename TIO, typename TST>
cudaError_t prompt_dims(const LinAttnArgs& a, cudaStream_t s) {
  if (a.dk == 64) return a.dv == 64 ? prompt_simt<TIO, TST, 64, 64>(a, s) : prompt_simt<TIO, TST, 64, 128>(a, s);
  return a.dv == 64 ? prompt_simt<TIO, TST, 128, 64>(a, s) : prompt_simt<TIO, TST, 128, 128>(a, s);
}

// ------------------------------------------------------------------ one token
// Eight columns a thread, DK / 8 lanes a row, NP rows a thread: a CTA updates NP * (1024 / DK) rows of
// one head's state.  The state is read and written once, straight through registers; k and q are the
// same for every row and come from L1 after the first.  Bound by HBM: 200 sequences of 16 fp32 heads 54 us
// = 6.4 TB/s, 0.95 of a plain copy's rate; 64 of 32 bf16 heads 24.6 us as a call, 0.81 (17 us replayed on one
// state, part of which stays in L2).  NP = 4 is the best where that counts (64 of 32 bf16 heads, states out of
// L2, 23 us; NP 1: 33, 2: 23.8, 8: 22.9 with fewer CTAs for small batches).
template <typename TIO, typename TST, int DK, int NP>
__global__ void __launch_bounds__(kThreads) linear_attn_step_kernel(LinStepArgs a) {
  constexpr int LPR = DK / 8, RPP = kThreads / LPR;  // lanes per row, rows per pass
  const int slabs = a.dv / (RPP * NP);
  const int slab = blockIdx.x % slabs, h = blockIdx.x / slabs % a.H, b = blockIdx.x / slabs / a.H;
  if (a.live != nullptr && __ldg(a.live + b) == 0) return;
  const int l = threadIdx.x % LPR, row0 = slab * RPP * NP + threadIdx.x / LPR;
  const int hk = h / (a.H / a.Hk);
  TST* sp = static_cast<TST*>(a.S) + (((size_t)b * a.H + h) * a.dv + row0) * DK + 8 * l;
  const TIO* vp = static_cast<const TIO*>(a.v) + b * a.v_stride + h * a.dv + row0;
  float s[NP][8], v[NP], k[8], q[8];
#pragma unroll
  for (int p = 0; p < NP; ++p) load_vec_rw<8>(sp + p * RPP * DK, s[p]);
  load_vec<8>(static_cast<const TIO*>(a.k) + b * a.k_stride + hk * DK + 8 * l, k);
  load_vec<8>(static_cast<const TIO*>(a.q) + b * a.q_stride + hk * DK + 8 * l, q);
#pragma unroll
  for (int p = 0; p < NP; ++p) v[p] = to_f32(vp[p * RPP]);
  const float al = __ldg(a.alpha + b * a.alpha_stride + h);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    float dot = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      s[p][c] = fmaf(v[p], k[c], al * s[p][c]);
      dot = fmaf(s[p][c], q[c], dot);
    }
    store_vec<8>(sp + p * RPP * DK, s[p]);
    dot = group_sum<LPR>(dot) * a.q_scale;
    if (l == 0)
      static_cast<TIO*>(a.out)[b * a.out_stride + h * a.dv + row0 + p * RPP] = from_f32<TIO>(dot);
  }
}

template <typename TIO, typename TST, int DK>
cudaError_t step_rows(const LinStepArgs& a, cudaStream_t s) {
  constexpr int RPP = kThreads * 8 / DK;
  constexpr int NP = 4;
  const long long grid = (long long)a.B * a.H * (a.dv / (RPP * NP));
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  linear_attn_step_kernel<TIO, TST, DK, NP><<<(unsigned)grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename TIO, typename TST>
cudaError_t step_dims(const LinStepArgs& a, cudaStream_t s) {
  return a.dk == 64 ? step_rows<TIO, TST, 64>(a, s) : step_rows<TIO, TST, 128>(a, s);
}

}  // namespace

int linear_attn_segment(int B, int T, int max_len, int H, int dk, int dv, int io) {
  (void)dk;
  const int sms = device_sm_count();
  if (io == TV_BF16) {
    // One CTA per SM walks whole (segment, head) units.  Measured on a GB300, in us: a unit costs 5 and
    // 3.2 a chunk of 128 tokens, in the pass over states alone 5 and 1.2; a launch 4, the scan 3 and
    // 0.4 a segment.  The cheapest cut of the longest prompt into equal pieces, or none.  (16 heads, one
    // prompt: 768 tokens 27 uncut and in six pieces; 4096 tokens 112 uncut, 39 in eight pieces.  32
    // heads, 32768 tokens: 848 uncut, 317 in four pieces.)
    // fp32 states take 1.2 to 1.3 times as long in both passes (third part of the keys) and are cut alike
    // (32768 tokens 1001 uncut, 401; 8 ragged prompts of up to 3001, 32 heads, 129 and 109).
    const int longest = (max_len + 127) / 128;
    // Prompts of one length run in rounds; of ragged ones the longest, which start first, or the sum counts,
    // each with a margin for CTAs that draw more than their share.
    auto pass = [&](int chunks, double each) {
      const double units = (double)H * std::max(B, (T / 128 + chunks - 1) / chunks), alone = 5 + each * chunks;
      if ((long long)B * max_len == T) return 4 + std::ceil(units / sms) * alone;
      return 4 + std::max(1.25 * alone, 1.15 * (units * 5 + each * H * (T / 128.0)) / sms);
    };
    auto cost = [&](int chunks) {
      if (chunks >= longest) return pass(chunks, 3.2);
      return pass(chunks, 3.2) + pass(chunks, 1.2) + 3 + 0.4 * ((longest + chunks - 1) / chunks);
    };
    int best = longest;
    for (int pieces = 2; pieces <= 64 && longest / pieces > 1; ++pieces) {
      const int chunks = (longest + pieces - 1) / pieces;
      if (cost(chunks) < 0.9 * cost(best)) best = chunks;
    }
    return best < longest ? best * 128 : 0;
  }
  // fp32: four CTAs for every SM, unless the prompts alone are near that.  Measured, in us, uncut and with two,
  // four and eight an SM: one prompt of 300 tokens, 4 heads 58, 30, 30, 30; 1000 tokens, 32 heads 185, 123,
  // 111, 120; 4096 tokens, 16 heads 742, 238, 237, 218; 32768 tokens, 8 heads 5900, 788, 794, 787; 8 ragged
  // prompts of up to 3001, 8 heads 544, 144, 134, 141; 4 prompts of 5000, 32 heads 1415, 1415, 1415, 1743.
  long long seg = ((long long)T * H * (dv / kRows) + 4 * sms - 1) / (4 * sms);
  seg = (seg + 63) / 64 * 64;
  return max_len > 3 * seg ? (int)seg : 0;
}

size_t linear_attn_workspace_size(int B, int T, int max_len, int H, int dk, int dv, int io) {
  if (max_len > T) max_len = T;
  const int seg = linear_attn_segment(B, T, max_len, H, dk, dv, io);
  if (seg == 0) return 0;
  const size_t segments = (size_t)B + T / seg;
  return segments * H * ((size_t)dv * dk + 4) * sizeof(float);
}

cudaError_t launch_linear_attn_scan(const LinAttnArgs& a, cudaStream_t s) {
  const int parts = (a.dk * a.dv / 4 + 255) / 256;
  const long long grid = (long long)a.B * a.H * parts;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (a.state == TV_BF16) linear_attn_scan_kernel<bf16><<<(unsigned)grid, 256, 0, s>>>(a, parts);
  else linear_attn_scan_kernel<float><<<(unsigned)grid, 256, 0, s>>>(a, parts);
  return cudaGetLastError();
}

// Whether walking token by token is cheaper than a chunk of 128 for every prompt.  Measured on a
// GB300, in us, U prompts x heads, T tokens: token by token 3 + 0.016 U + T (0.12 + 0.002 U), in chunks
// 6 + 5.5 a round of one unit on every SM.  (16 heads, one prompt: 8 tokens 4.4 and 11.6; 64 tokens
// 11.7 and 12.4.  32 prompts of 32 heads: 4 tokens 27 and 44; 16 tokens 50 and 44.)
static bool short_prompts(const LinAttnArgs& a) {
  if (a.T == 0) return true;
  if (a.max_len > 128 || a.seg_len > 0) return false;
  const double units = (double)a.B * a.H, sms = device_sm_count();
  return 3 + 0.016 * units + a.max_len * (0.12 + 0.002 * units) < 6 + 5.5 * (long long)((units + sms - 1) / sms);
}

cudaError_t launch_linear_attn_prompt(const LinAttnArgs& a, cudaStream_t s) {
  if (a.io == TV_BF16 && !short_prompts(a)) return launch_linear_attn_tc(a, s);
  if (a.io == TV_F32) return prompt_dims<float, float>(a, s);
  return a.state == TV_BF16 ? prompt_dims<bf16, bf16>(a, s) : prompt_dims<bf16, float>(a, s);
}

cudaError_t launch_linear_attn_step(const LinStepArgs& a, cudaStream_t s) {
  if (a.io == TV_F32) return step_dims<float, float>(a, s);
  return a.state == TV_BF16 ? step_dims<bf16, bf16>(a, s) : step_dims<bf16, float>(a, s);
}

}  // namespace tv
