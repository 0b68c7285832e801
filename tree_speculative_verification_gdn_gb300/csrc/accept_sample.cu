// Acceptance of draft trees by probabilities, and the draw of the token after them.
//
// At a node the tokens refused one after another leave R_k = max(R_{k-1} - M_{k-1} q, 0), M_k = sum R_k, of the target's
// row p.  Since max(max(x - y, 0) - z, 0) = max(x - y - z, 0) for y, z >= 0, that is R_k = max(p - A_k q, 0) with
// A_k = M_0 + ... + M_{k-1}: one scalar stands for the state, and a refusal costs one pass over the rows p and q.
// Where q is not known, refused tokens are left out of p instead, and no pass is needed before the draw.
//
// A token next to a border decides, so sums are carried as two floats each (p - A q by exact differences and products,
// sums by exact additions, about 2^-46), joined in doubles; a double per element would cost more than the row's bytes:
// this chip adds two doubles a clock on an SM.
//
// A cluster of eight CTAs takes a sequence, each the eighth part of a row, each of its 16 warps a run of that part.  Every
// CTA walks the tree by itself on the same sums.  The draw finds the warp's run from the 128 sums, and that warp
// walks its run again, which lies in L2.  Bound by the latency of a pass where sequences are few, by HBM otherwise.
#include "tv_common.cuh"
#include "tv_internal.h"
#include "tv_tc.cuh"

namespace tv {
namespace {

constexpr int kParts = 8;
constexpr int kWarps = 16;
constexpr int kRuns = kParts * kWarps;

// hi + lo, lo far below hi
struct Pair {
  float hi, lo;
};
// acc + (x.hi + x.lo), the addition's error kept
__device__ __forceinline__ void add(Pair& acc, Pair x) {
  const float t = __fadd_rn(acc.hi, x.hi);
  const float b = __fsub_rn(t, acc.hi);
  const float e = __fadd_rn(__fsub_rn(acc.hi, __fsub_rn(t, b)), __fsub_rn(x.hi, b));
  acc.hi = t;
  acc.lo = __fadd_rn(acc.lo, __fadd_rn(e, x.lo));
}
// max(p - A q, 0)
__device__ __forceinline__ Pair left_of(float p, float q, Pair A) {
  const float y = __fmul_rn(A.hi, q);
  const float ye = __fadd_rn(__fmaf_rn(A.hi, q, -y), __fmul_rn(A.lo, q));
  const float d = __fsub_rn(p, y);
  const float b = __fsub_rn(d, p);
  const float e = __fsub_rn(__fsub_rn(__fsub_rn(p, __fsub_rn(d, b)), __fadd_rn(y, b)), ye);
  return __fadd_rn(d, e) > 0.f ? Pair{d, e} : Pair{0.f, 0.f};
}
__device__ __forceinline__ double whole(Pair x) { return (double)x.hi + (double)x.lo; }

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_st_f64(uint32_t caddr, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(caddr), "d"(v) : "memory");
}

template <typename T>
struct Rows {  // rows p and q of a node, in vectors of 16 bytes from the boundary at or before their start
  static constexpr int VE = 16 / (int)sizeof(T);
  const T* p;
  const T* q;  // nullptr: not known
  int V, phase;
  __device__ static void vector(const T* row, int e, int V, float* x) {  // elements e .. e + VE - 1, zero outside
    if (e >= 0 && e + VE <= V) {
      load_vec<VE>(row + e, x);
    } else {
#pragma unroll
      for (int i = 0; i < VE; ++i) x[i] = e + i >= 0 && e + i < V ? to_f32(row[e + i]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < VE; ++i) x[i] = fmaxf(x[i], 0.f);  // NaN too
  }
};

template <typename T>
__global__ void __cluster_dims__(kParts, 1, 1) __launch_bounds__(kWarps * 32) accept_sample_kernel(SampleArgs a) {
  constexpr int VE = Rows<T>::VE;
  __shared__ int par[TV_MAX_NODES], tok[TV_MAX_NODES], path[TV_MAX_NODES], refused[TV_MAX_NODES];
  __shared__ float u[TV_MAX_NODES], pt[TV_MAX_NODES], qt[TV_MAX_NODES];
  __shared__ double sums[2][kRuns];
  const int b = blockIdx.x / kParts, rank = (int)cluster_ctarank();
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int N = a.N, V = a.V;
  cluster_arrive();  // no CTA writes to another's sums before that one runs
  const T* target = static_cast<const T*>(a.target) + (long long)b * N * V;
  const T* draft = a.draft != nullptr ? static_cast<const T*>(a.draft) + (long long)b * N * V : nullptr;
  bool bad = false;
  for (int i = tid; i < N; i += blockDim.x) {
    const int p = a.parents[(long long)b * N + i], x = a.tokens[(long long)b * N + i];
    par[i] = p, tok[i] = x;
    u[i] = a.uniforms[(long long)b * N + i];
    const bool ok = p >= 0 && p < i && x >= 0 && x < V;
    pt[i] = ok ? fmaxf(to_f32(target[(long long)p * V + x]), 0.f) : 0.f;
    qt[i] = ok && draft != nullptr ? fmaxf(to_f32(draft[(long long)p * V + x]), 0.f) : 0.f;
    bad |= p < -1 || p >= i;
  }
  bad = __syncthreads_or(bad);
  cluster_wait();
  auto fail = [&](int st) {
    if (rank != 0) return;
    for (int r = tid; r < a.Lmax; r += blockDim.x) a.path[(long long)b * a.Lmax + r] = -1;
    if (tid == 0) a.len[b] = 0, a.next_token[b] = -1, a.err[b] = st;
  };
  if (bad) return fail(TV_ERR_BAD_TREE);

  int parity = 0;
  int count_refused = 0;  // tokens left out of p (q not known)
  Rows<T> r;
  r.V = V;
  int v0 = 0, v1 = 0;  // this warp's run of vectors
  auto rows_of = [&](int node) {
    r.p = target + (long long)node * V;
    r.q = draft != nullptr ? draft + (long long)node * V : nullptr;
    r.phase = (int)((reinterpret_cast<uintptr_t>(r.p) & 15u) / sizeof(T));
    const int vecs = (V + r.phase + VE - 1) / VE;
    const int per = ((vecs + kParts - 1) / kParts + kWarps - 1) / kWarps;
    v0 = min((rank * kWarps + warp) * per, vecs), v1 = min(v0 + per, vecs);
  };
  // whether this warp's run holds a token that was left out of p
  auto any_refused = [&]() -> bool {
    bool in = false;
    for (int k = lane; k < count_refused; k += 32) {
      const int at = refused[k] + r.phase;
      in |= at >= v0 * VE && at < v1 * VE;
    }
    return __any_sync(0xffffffffu, in);
  };
  // R of vector j, as pairs
  auto left = [&](int j, Pair A, bool use_q, bool some, Pair* x) {
    const int e = j * VE - r.phase;
    float p[VE], q[VE];
    Rows<T>::vector(r.p, e, V, p);
    if (use_q) Rows<T>::vector(r.q, e, V, q);
#pragma unroll
    for (int i = 0; i < VE; ++i) x[i] = use_q ? left_of(p[i], q[i], A) : Pair{p[i], 0.f};
    for (int k = 0; some && k < count_refused; ++k) {
      const int at = refused[k] - e;
#pragma unroll
      for (int i = 0; i < VE; ++i)
        if (i == at) x[i] = Pair{0.f, 0.f};
    }
  };
  // sum R; every run's own sum in sums[parity]
  auto pass = [&](double Ad) -> double {
    const Pair A{(float)Ad, (float)(Ad - (double)(float)Ad)};
    const bool use_q = Ad != 0.0, some = any_refused();
    Pair acc{0.f, 0.f};
#pragma unroll 4
    for (int j = v0 + lane; j < v1; j += 32) {
      Pair x[VE];
      left(j, A, use_q, some, x);
#pragma unroll
      for (int i = 0; i < VE; ++i) add(acc, x[i]);
    }
    const double run = warp_sum(whole(acc));
    parity ^= 1;
    if (lane < kParts) cluster_st_f64(cluster_map(smem_addr(&sums[parity][rank * kWarps + warp]), lane), run);
    cluster_sync();
    double m = 0.0;
#pragma unroll
    for (int k = 0; k < kRuns / 32; ++k) m += sums[parity][lane * (kRuns / 32) + k];
    return warp_sum(m);
  };

  int node = 0, count = 1;
  if (tid == 0) path[0] = 0;
  double A = 0.0, mass = 1.0;  // of the tokens refused at this node
  bool have = false;           // mass is the last pass's sum of R
  rows_of(0);
  while (count < a.Lmax) {
    int went = -1;
    for (int base = (node + 1) & ~31; base < N && went < 0; base += 32) {
      unsigned kids = __ballot_sync(0xffffffffu, base + lane < N && base + lane > node && par[base + lane] == node);
      while (kids != 0 && went < 0) {
        const int c = base + __ffs(kids) - 1;
        kids &= kids - 1;
        if (draft != nullptr) {
          const double rx = fmax((double)pt[c] - A * (double)qt[c], 0.0);
          if ((double)u[c] * (double)qt[c] * mass < rx) {
            went = c;
          } else {
            A += mass;
            mass = pass(A);
            have = true;
            if (!(mass > 0.0)) A = 0.0, mass = 1.0, have = false;
          }
        } else {
          double rx = (double)pt[c];
          for (int k = 0; k < count_refused; ++k)
            if (refused[k] == tok[c]) rx = 0.0;
          if ((double)u[c] * mass < rx) {
            went = c;
          } else {
            mass -= rx;
            __syncthreads();  // every thread is done with the list
            if (tid == 0) refused[count_refused] = tok[c];
            __syncthreads();
            ++count_refused;
          }
        }
      }
    }
    if (went < 0) break;
    node = went;
    if (tid == 0) path[count] = node;
    ++count;
    A = 0.0, mass = 1.0, have = false, count_refused = 0;
    rows_of(node);
  }
  // the token after the accepted ones
  if (!have) mass = pass(A);
  if (!(mass > 0.0) && (A != 0.0 || count_refused != 0)) {
    A = 0.0, count_refused = 0;
    mass = pass(A);
  }
  if (!(mass > 0.0)) return fail(TV_ERR_BAD_PROBS);
  const double want = (double)u[0] * mass;
  double mine[kRuns / 32], before = 0.0;
#pragma unroll
  for (int k = 0; k < kRuns / 32; ++k) before += mine[k] = sums[parity][lane * (kRuns / 32) + k];
  const double own_sum = before;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double x = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += x;
  }
  before -= own_sum;  // of the runs in front of this lane's four
  int run = kRuns, last = -1;
  double ahead = 0.0, upto = before;
#pragma unroll
  for (int k = 0; k < kRuns / 32; ++k) {
    if (mine[k] > 0.0) last = lane * (kRuns / 32) + k;
    if (run == kRuns && mine[k] > 0.0 && upto + mine[k] > want) run = lane * (kRuns / 32) + k, ahead = upto;
    upto += mine[k];
  }
  const unsigned found = __ballot_sync(0xffffffffu, run < kRuns);
  if (found != 0) {
    run = __shfl_sync(0xffffffffu, run, __ffs(found) - 1);
    ahead = __shfl_sync(0xffffffffu, ahead, __ffs(found) - 1);
  } else {  // rounding, or a number past 1: the last token with a probability
    run = __reduce_max_sync(0xffffffffu, last);
    ahead = 0.0;
  }
  if (run == rank * kWarps + warp) {
    const Pair Ap{(float)A, (float)(A - (double)(float)A)};
    const bool some = any_refused();
    int token = -1, last_token = -1;
    for (int j0 = v0; j0 < v1 && token < 0; j0 += 32) {
      const int j = j0 + lane;
      Pair x[VE];
#pragma unroll
      for (int i = 0; i < VE; ++i) x[i] = Pair{0.f, 0.f};
      if (j < v1) left(j, Ap, A != 0.0, some, x);
      double sum = 0.0;
      int positive = -1;
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        sum += whole(x[i]);
        if (x[i].hi > 0.f || x[i].lo > 0.f) positive = j * VE - r.phase + i;
      }
      double to = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, to, o);
        if (lane >= o) to += y;
      }
      const double from = ahead + (to - sum);
      int hit = -1;
      if (found != 0) {
        double run_sum = from;
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          const double v = whole(x[i]);
          run_sum += v;
          if (hit < 0 && v > 0.0 && run_sum > want) hit = j * VE - r.phase + i;
        }
      }
      const unsigned hits = __ballot_sync(0xffffffffu, hit >= 0);
      if (hits != 0) token = __shfl_sync(0xffffffffu, hit, __ffs(hits) - 1);
      last_token = max(last_token, __reduce_max_sync(0xffffffffu, positive));
      ahead += __shfl_sync(0xffffffffu, to, 31);
    }
    if (lane == 0) a.next_token[b] = token >= 0 ? token : last_token;
  }
  if (rank == 0) {
    __syncthreads();
    for (int i = tid; i < a.Lmax; i += blockDim.x) a.path[(long long)b * a.Lmax + i] = i < count ? path[i] : -1;
    if (tid == 0) a.len[b] = count, a.err[b] = 0;
  }
}

}  // namespace

cudaError_t launch_accept_sample(const SampleArgs& a, cudaStream_t s) {
  if (a.probs == TV_F32) accept_sample_kernel<float><<<a.B * kParts, kWarps * 32, 0, s>>>(a);
  else accept_sample_kernel<bf16><<<a.B * kParts, kWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace tv
