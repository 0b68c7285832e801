// Acceptance of draft trees by probabilities, and the draw of the token after them.
//
// At a node the tokens refused one after another leave R_k = max(R_{k-1} - M_{k-1} q, 0), M_k = sum R_k, of the target's
// row p.  Since max(max(x - y, 0) - z, 0) = max(x - y - z, 0) for y, z >= 0, that is R_k = max(p - A_k q, 0) with
// A_k = M_0 + ... + M_{k-1}: one scalar stands for the state, and a refusal costs one pass over the rows p and q.
// Where q is not known, refused tokens are left out of p instead, and no pass is needed before the draw.
//
// A token next to a border decides, so sums are carried as two floats each: p - A q by exact differences and products, sums
// by exact additions, about 2^-46.  Doubles would cost more than the row's bytes, two additions a clock on an SM, and their
// latency most of a short call: 64 chains of four tokens, 131072 values of fp32, took 76 us in doubles, 25 with pairs for
// the values alone, 17 with pairs throughout.
//
// A cluster of up to eight CTAs takes a sequence, each an equal part of a row, each of its 16 warps a run of that part.
// Every CTA walks the tree by itself on the same sums.  The draw finds the warp's run from the runs' sums, and its
// CTA cuts that again, which lies in L2.  Bound by the latency of a pass where sequences are few, by HBM otherwise.
#include "tv_common.cuh"
#include "tv_internal.h"
#include "tv_tc.cuh"

namespace tv {
namespace {

constexpr int kWarps = 16;

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
__device__ __forceinline__ Pair sum_of(Pair a, Pair b) {  // with lo small against hi again
  add(a, b);
  const float t = __fadd_rn(a.hi, a.lo);
  return Pair{t, __fsub_rn(a.lo, __fsub_rn(t, a.hi))};
}
__device__ __forceinline__ Pair product(float f, Pair x) {
  const float y = __fmul_rn(f, x.hi);
  return Pair{y, __fadd_rn(__fmaf_rn(f, x.hi, -y), __fmul_rn(f, x.lo))};
}
__device__ __forceinline__ bool less(Pair a, Pair b) {
  const float d = __fsub_rn(a.hi, b.hi);
  const float t = __fsub_rn(d, a.hi);
  const float e = __fsub_rn(__fsub_rn(a.hi, __fsub_rn(d, t)), __fadd_rn(b.hi, t));
  return __fadd_rn(d, __fadd_rn(e, __fsub_rn(a.lo, b.lo))) < 0.f;
}
// max(p - A q, 0)
__device__ __forceinline__ Pair left_of(float p, float q, Pair A) {
  const Pair y = product(q, A);
  const float d = __fsub_rn(p, y.hi);
  const float b = __fsub_rn(d, p);
  const float e = __fsub_rn(__fsub_rn(__fsub_rn(p, __fsub_rn(d, b)), __fadd_rn(y.hi, b)), y.lo);
  return __fadd_rn(d, e) > 0.f ? Pair{d, e} : Pair{0.f, 0.f};
}
// The first refusal at a node, A = 1: where p > q the error of p - q takes two steps, and elsewhere nothing is left.
__device__ __forceinline__ Pair left_of(float p, float q) {
  const float d = __fsub_rn(p, q);
  const float e = __fsub_rn(__fsub_rn(p, d), q);
  return d > 0.f ? Pair{d, e} : Pair{0.f, 0.f};
}
// Two sums side by side in packed registers.
struct Pair2 {
  float2 hi, lo;
};
__device__ __forceinline__ float2 minus(float2 a, float2 b) { return __ffma2_rn(b, make_float2(-1.f, -1.f), a); }
__device__ __forceinline__ void add(Pair2& acc, Pair x, Pair y) {
  const float2 v = make_float2(x.hi, y.hi);
  const float2 t = __fadd2_rn(acc.hi, v);
  const float2 b = minus(t, acc.hi);
  const float2 e = __fadd2_rn(minus(acc.hi, minus(t, b)), minus(v, b));
  acc.hi = t;
  acc.lo = __fadd2_rn(acc.lo, __fadd2_rn(e, make_float2(x.lo, y.lo)));
}

// Over the lanes up to this one.
template <int LANES>
__device__ __forceinline__ Pair warp_scan(Pair x) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) {
    const Pair y{__shfl_up_sync(0xffffffffu, x.hi, o), __shfl_up_sync(0xffffffffu, x.lo, o)};
    if ((int)(threadIdx.x % 32) >= o) x = sum_of(y, x);
  }
  return x;
}
__device__ __forceinline__ Pair of_lane(Pair x, int lane) {
  return Pair{__shfl_sync(0xffffffffu, x.hi, lane), __shfl_sync(0xffffffffu, x.lo, lane)};
}
// The first lane's, in every lane: add() rounds lo by the order of its two numbers, so that the lanes of a butterfly end up
// to a rounding of lo apart, and a CTA that decided on another lane's number might walk or draw apart from its cluster.
__device__ __forceinline__ Pair warp_sum(Pair x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    add(x, Pair{__shfl_xor_sync(0xffffffffu, x.hi, o), __shfl_xor_sync(0xffffffffu, x.lo, o)});
  return of_lane(x, 0);
}
// Of the lane before, 0 in the first.
__device__ __forceinline__ Pair before_lane(Pair x) {
  const Pair y{__shfl_up_sync(0xffffffffu, x.hi, 1), __shfl_up_sync(0xffffffffu, x.lo, 1)};
  return threadIdx.x % 32 == 0 ? Pair{0.f, 0.f} : y;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_st_pair(uint32_t caddr, Pair v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(caddr), "f"(v.hi), "f"(v.lo) : "memory");
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
  }
};

// What the walk, one warp's, asks of the others.
struct Ask {
  int node;
  Pair A;
  int refused;  // tokens left out
  int draw;     // 0: another pass; 1: the draw, from the last pass's sums; < 0: a status to report
  int run;      // the draw's run; the sum in front of it, and the number to pass (none: the last token with any)
  Pair ahead, want;
  int found;
};

// kParts CTAs a sequence.
template <typename T, int kParts>
__global__ void __cluster_dims__(kParts, 1, 1) __launch_bounds__(kWarps * 32, 2) accept_sample_kernel(SampleArgs a) {
  constexpr int VE = Rows<T>::VE;
  constexpr int kRuns = kParts * kWarps;
  constexpr int kOwn = kRuns >= 32 ? kRuns / 32 : 1;  // sums of a lane of the walk's warp; the upper lanes may have none
  __shared__ int par[TV_MAX_NODES], tok[TV_MAX_NODES], path[TV_MAX_NODES], refused[TV_MAX_NODES];
  __shared__ float u[TV_MAX_NODES], pt[TV_MAX_NODES], qt[TV_MAX_NODES];
  __shared__ Pair sums[2][kRuns];
  __shared__ Ask ask;
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

  // The walk: the whole of warp 0 keeps the same state.
  int node = 0, count = 1, at = 0;     // at: the last child looked at
  int left_out = 0, parity = 0;
  Pair A{0.f, 0.f}, mass{1.f, 0.f};
  bool have = false;  // mass is the sum of the last pass
  if (tid == 0) path[0] = 0;
  // On to the next pass, or to the draw.
  auto walk = [&]() {
    while (count < a.Lmax) {
      int went = -1;
      for (int base = (at + 1) & ~31; base < N && went < 0; base += 32) {
        unsigned kids = __ballot_sync(0xffffffffu, base + lane < N && base + lane > at && par[base + lane] == node);
        while (kids != 0) {
          const int c = base + __ffs(kids) - 1;
          kids &= kids - 1;
          if (draft != nullptr) {
            if (less(product(u[c], product(qt[c], mass)), left_of(pt[c], qt[c], A))) {
              went = c;
              break;
            }
            at = c;
            A = sum_of(A, mass);
            ask.draw = 0;
            return;  // for the sum of what is left
          }
          bool twice = false;
          for (int k = lane; k < left_out; k += 32) twice |= refused[k] == tok[c];
          const float rx = __any_sync(0xffffffffu, twice) ? 0.f : pt[c];
          if (less(product(u[c], mass), Pair{rx, 0.f})) {
            went = c;
            break;
          }
          mass = sum_of(mass, Pair{-rx, 0.f});
          if (lane == 0) refused[left_out] = tok[c];
          __syncwarp();
          ++left_out;
        }
      }
      if (went < 0) break;
      node = at = went;
      if (lane == 0) path[count] = node;
      ++count;
      A = Pair{0.f, 0.f}, mass = Pair{1.f, 0.f}, have = false, left_out = 0;
    }
    ask.draw = have ? 1 : 0;
    at = N;  // no child is left to look at
  };
  // With the last pass's sums: goes on, or finds the run that the drawn token lies in.
  auto take = [&]() {
    Pair own[kOwn], all{0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      own[k] = lane * kOwn + k < kRuns ? sums[parity][lane * kOwn + k] : Pair{0.f, 0.f};
      all = sum_of(all, own[k]);
    }
    const Pair upto = warp_scan<32>(all);
    mass = of_lane(upto, 31);
    have = true;
    if (!(mass.hi > 0.f)) {
      if (at < N) {  // nothing is left: the next child is held against p again
        A = Pair{0.f, 0.f}, mass = Pair{1.f, 0.f}, have = false;
      } else if (A.hi != 0.f || left_out != 0) {
        A = Pair{0.f, 0.f}, left_out = 0;
        ask.draw = 0;
        return;
      } else {
        ask.draw = TV_ERR_BAD_PROBS;
        return;
      }
    }
    if (at < N) walk();
    if (ask.draw == 0) {
      if (at < N || !have) return;
      ask.draw = 1;
    }
    const Pair want = product(u[0], mass);
    Pair to = before_lane(upto), ahead{0.f, 0.f};
    int run = kRuns, last = -1;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      const Pair next = sum_of(to, own[k]);
      if (own[k].hi > 0.f) last = lane * kOwn + k;
      if (run == kRuns && own[k].hi > 0.f && less(want, next)) run = lane * kOwn + k, ahead = to;
      to = next;
    }
    const unsigned found = __ballot_sync(0xffffffffu, run < kRuns);
    if (found != 0) {
      run = __shfl_sync(0xffffffffu, run, __ffs(found) - 1);
      ahead = of_lane(ahead, __ffs(found) - 1);
    } else {  // rounding, or a number past 1: the last token with a probability
      run = __reduce_max_sync(0xffffffffu, last);
    }
    ask.run = run, ask.ahead = ahead, ask.want = want, ask.found = found != 0;
  };
  auto tell = [&]() { ask.node = node, ask.refused = left_out, ask.A = A; };

  Rows<T> r;
  r.V = V;
  int v0 = 0, v1 = 0;  // this warp's run of vectors
  bool some = false;   // it holds a token that was left out of p
  Pair Ap{0.f, 0.f};
  int form = 0;        // of what is left: p, p - q, p - A q
  auto listen = [&]() {
    r.p = target + (long long)ask.node * V;
    r.q = draft != nullptr ? draft + (long long)ask.node * V : nullptr;
    r.phase = (int)((reinterpret_cast<uintptr_t>(r.p) & 15u) / sizeof(T));
    const int vecs = (V + r.phase + VE - 1) / VE;
    const int per = ((vecs + kParts - 1) / kParts + kWarps - 1) / kWarps;
    v0 = min((rank * kWarps + warp) * per, vecs), v1 = min(v0 + per, vecs);
    bool in = false;
    for (int k = lane; k < ask.refused; k += 32) {
      const int e = refused[k] + r.phase;
      in |= e >= v0 * VE && e < v1 * VE;
    }
    some = __any_sync(0xffffffffu, in);
    Ap = ask.A;
    form = Ap.hi == 0.f ? 0 : Ap.hi == 1.f && Ap.lo == 0.f ? 1 : 2;
  };
  // R of vector j, as pairs; negative probabilities and NaN count as 0
  auto left = [&](int form, int j, Pair* x) {
    const int e = j * VE - r.phase;
    float p[VE], q[VE];
    Rows<T>::vector(r.p, e, V, p);
    if (form != 0) Rows<T>::vector(r.q, e, V, q);
#pragma unroll
    for (int i = 0; i < VE; ++i)
      x[i] = form == 0 ? Pair{fmaxf(p[i], 0.f), 0.f}
             : form == 1 ? left_of(p[i], fmaxf(q[i], 0.f)) : left_of(p[i], fmaxf(q[i], 0.f), Ap);
    for (int k = 0; some && k < ask.refused; ++k) {
      const int at = refused[k] - e;
#pragma unroll
      for (int i = 0; i < VE; ++i)
        if (i == at) x[i] = Pair{0.f, 0.f};
    }
  };
  // The sum of a run, in each of the three forms a loop of its own.
  auto run_sum = [&]() -> Pair {
    auto loop = [&](auto form) -> Pair {
      Pair2 acc{make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 4
      for (int j = v0 + lane; j < v1; j += 32) {
        Pair x[VE];
        left(form(), j, x);
#pragma unroll
        for (int i = 0; i < VE; i += 2) add(acc, x[i], x[i + 1]);
      }
      return warp_sum(sum_of(Pair{acc.hi.x, acc.lo.x}, Pair{acc.hi.y, acc.lo.y}));
    };
    if (form == 0) return loop([] { return 0; });
    return form == 1 ? loop([] { return 1; }) : loop([] { return 2; });
  };

  if (warp == 0) {
    if (bad) {
      ask.draw = TV_ERR_BAD_TREE;
    } else {
      walk();
      tell();
    }
  }
  __syncthreads();
  // Every CTA of the cluster makes the same passes, on the same sums.
  while (ask.draw == 0) {
    listen();
    const Pair acc = run_sum();
    parity ^= 1;
    if (lane < kParts) cluster_st_pair(cluster_map(smem_addr(&sums[parity][rank * kWarps + warp]), lane), acc);
    cluster_sync();
    if (warp == 0) {
      take();
      tell();
    }
    __syncthreads();
  }
  if (ask.draw < 0) {
    if (rank == 0) {
      for (int i = tid; i < a.Lmax; i += blockDim.x) a.path[(long long)b * a.Lmax + i] = -1;
      if (tid == 0) a.len[b] = 0, a.next_token[b] = -1, a.err[b] = ask.draw;
    }
    return;
  }
  if (rank == 0 && warp == 0) {
    for (int i = lane; i < a.Lmax; i += 32) a.path[(long long)b * a.Lmax + i] = i < count ? path[i] : -1;
    if (lane == 0) a.len[b] = count, a.err[b] = 0;
  }
  // The drawn token: the run's CTA cuts it among its warps in turn, and finds the warp whose part passes the number.
  if (ask.run / kWarps != rank) return;
  listen();
  {
    const int vecs = (V + r.phase + VE - 1) / VE;
    const int per = ((vecs + kParts - 1) / kParts + kWarps - 1) / kWarps, cut = (per + kWarps - 1) / kWarps;
    const int r0 = min(ask.run * per, vecs), r1 = min(r0 + per, vecs);
    v0 = min(r0 + warp * cut, r1), v1 = min(v0 + cut, r1);
    some = ask.refused > 0;
  }
  __shared__ Pair parts[kWarps];
  const Pair acc = run_sum();
  if (lane == 0) parts[warp] = acc;
  __syncthreads();
  const Pair want = ask.want;
  if (warp == 0) {
    const Pair own = lane < kWarps ? parts[lane] : Pair{0.f, 0.f};
    const Pair scan = warp_scan<kWarps>(own);
    const Pair to = sum_of(ask.ahead, scan), from = sum_of(ask.ahead, before_lane(scan));
    const unsigned hits = __ballot_sync(0xffffffffu, ask.found != 0 && own.hi > 0.f && less(want, to));
    const unsigned any = __ballot_sync(0xffffffffu, own.hi > 0.f);
    // no part passes it after all, by rounding: the last token of the last part with any
    const int part = hits != 0 ? __ffs(hits) - 1 : 31 - __clz((int)any);
    const Pair ahead = of_lane(from, part);
    __syncwarp();
    if (lane == 0) ask.run = part, ask.ahead = ahead, ask.found = hits != 0;
  }
  __syncthreads();
  if (ask.run != warp) return;
  // Four steps of 32 vectors at a time, so that their loads are under way together; the step that passes the number from
  // its lanes' sums, then the lane and the element.
  Pair ahead = ask.ahead;
  int token = -1, last_token = -1;
  for (int j0 = v0; j0 < v1 && token < 0; j0 += 128) {
    Pair sum[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int j = j0 + s * 32 + lane;
      Pair x[VE];
#pragma unroll
      for (int i = 0; i < VE; ++i) x[i] = Pair{0.f, 0.f};
      if (j < v1) left(form, j, x);
      sum[s] = Pair{0.f, 0.f};
      int positive = -1;
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        if (x[i].hi > 0.f) positive = j * VE - r.phase + i;
        add(sum[s], x[i]);
      }
      last_token = max(last_token, __reduce_max_sync(0xffffffffu, positive));
    }
    if (ask.found == 0) continue;
#pragma unroll 1
    for (int s = 0; s < 4 && token < 0; ++s) {
      const Pair scan = warp_scan<32>(s == 0 ? sum[0] : s == 1 ? sum[1] : s == 2 ? sum[2] : sum[3]);
      if (__any_sync(0xffffffffu, less(want, sum_of(ahead, scan)))) {
        const int j = j0 + s * 32 + lane;
        Pair x[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i) x[i] = Pair{0.f, 0.f};
        if (j < v1) left(form, j, x);
        Pair to = sum_of(ahead, before_lane(scan));
        int hit = -1;
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          to = sum_of(to, x[i]);
          if (hit < 0 && x[i].hi > 0.f && less(want, to)) hit = j * VE - r.phase + i;
        }
        const unsigned hits = __ballot_sync(0xffffffffu, hit >= 0);
        if (hits != 0) token = __shfl_sync(0xffffffffu, hit, __ffs(hits) - 1);
      }
      ahead = sum_of(ahead, of_lane(scan, 31));
    }
  }
  if (lane == 0) a.next_token[b] = token >= 0 ? token : last_token;
}

}  // namespace

namespace {

template <typename T>
cudaError_t go(const SampleArgs& a, cudaStream_t s) {
  // As many CTAs a sequence as are resident at once: two on an SM.
  constexpr int kThreads = kWarps * 32;
  const int room = 2 * device_sm_count();
  if (a.B * 8LL <= room) accept_sample_kernel<T, 8><<<a.B * 8, kThreads, 0, s>>>(a);
  else if (a.B * 4LL <= room) accept_sample_kernel<T, 4><<<a.B * 4, kThreads, 0, s>>>(a);
  else if (a.B * 2LL <= room) accept_sample_kernel<T, 2><<<a.B * 2, kThreads, 0, s>>>(a);
  else accept_sample_kernel<T, 1><<<a.B, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_accept_sample(const SampleArgs& a, cudaStream_t s) {
  return a.probs == TV_F32 ? go<float>(a, s) : go<bf16>(a, s);
}

}  // namespace tv
