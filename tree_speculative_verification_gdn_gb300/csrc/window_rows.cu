// Windowed attention of few query rows -- single tokens, short drafted chains -- over long contexts.
//
// The rows of a sequence and KV head, (new token, query head of the group), are at most 16, and every visible key and
// value is read once for all of them: bound by HBM.  The visible pages of all sequences and KV heads, one behind the
// other, are dealt out to the grid in equal runs, so that ragged lengths and few sequences spread alike.  A CTA's four warps
// take the pages of its run in turn, each with its own ring of copies in flight, its own running maximum, sum and
// output; no two warps meet inside a run.  Scores and outputs go through m16n8k16 products: at 16 rows a page, the
// matrix units are idle nine tenths of the time, and their registers need no detour through tensor memory.  Rows of
// a page that no token sees are not read; the copy fills them with zeros.
//
// A (sequence, KV head) that lies in several CTAs' runs leaves maximum, sum and unnormalised output per CTA in the
// workspace; the last of them to finish joins them in the order of the runs, so the result does not depend on which that is.
// So does a CTA with the parts of a long run.
//
// 64 sequences behind 8192 tokens, 16 heads on 4 of 128 columns: 1.07 GB in 170 us, none of it in L2, 6.3 TB/s.  One sequence
// behind 4096: 15 us, the plan, a run's copies and the joining one behind the other.
#include "tv_async.cuh"
#include "window_attn.cuh"

namespace tv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;      // query rows of a unit
constexpr int kWhole = 16;     // pages of a sequence and head that are never cut
constexpr int kLeast = 8;      // pages a run, at least: below, joining costs more than the pages
// Pages after which a CTA joins its warps' outputs, in the workspace: the matrix units cut what they add to a sum, which left
// outputs 5e-3 short with 2^20 keys a warp.  Parts of 2^15 keys a warp, joined in fp32, lose 2e-4, a tenth of the
// store's rounding.
constexpr int kSpan = 8192;
constexpr float kRaise = 8.f;  // the running maximum is raised only by more than this (log2): sums grow by 2^8 at most

constexpr int per_sm(int hd) { return hd == 256 ? 1 : hd == 128 ? 2 : 3; }

template <int HD>
struct Shape {
  static constexpr int kStages = HD == 64 ? 4 : 3;
  static constexpr int kPage = 16 * HD * 2;  // bytes of one page of keys (or values) of a head
  static constexpr int kRing = kWarps * kStages * 2 * kPage;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16-byte chunk c of a row, its low three bits turned by the row: eight rows of one chunk meet all banks.
template <int HD>
__device__ __forceinline__ uint32_t chunk_at(int row, int c) {
  return row * (HD * 2) + ((c ^ (row & 7)) << 4);
}

template <int HD>
__global__ void __launch_bounds__(kThreads, per_sm(HD))
    window_rows_kernel(WinAttnArgs a, const long long* cost, float* slots, int* arrived) {
  using S = Shape<HD>;
  constexpr int kSlot = kRows * (HD + 4);  // floats: outputs, then (maximum, sum) per row, twice: to read and to write
  constexpr int CH = HD / 8;                 // 16-byte chunks of a row
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* sQ = smem;                          // kRows rows
  unsigned char* ring = smem + kRows * HD * 2;
  __shared__ int s_last;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int G = a.Hq / a.Hkv;

  wait_for_plan();
  Run run;
  if (!find_run<kThreads>(a, cost, kLeast, run)) return;
  int b = run.b, start = run.start;
  long long base = run.base;
  const long long per = run.per, x0 = run.x0, x1 = run.x1;
  Seen q = seen_by(a, run.P, run.n);

  const float scale = a.sm_scale * 1.4426950408889634f;
  const uint32_t my_ring = smem_addr(ring) + warp * (S::kStages * 2 * S::kPage);
  bool used = false;
  for (long long x = x0; x < x1;) {
    if (x - base >= (long long)q.pages * a.Hkv) {
      base += (long long)q.pages * a.Hkv;
      while (cost[++b] == 0) {}
      start = a.cu != nullptr ? a.cu[b] : b;
      q = seen_by(a, a.prefix_len[b], a.cu != nullptr ? a.cu[b + 1] - start : 1);
    }
    const int kvh = (int)quotient(x - base, q.pages);
    const long long u0 = base + (long long)kvh * q.pages, u1 = u0 + q.pages;
    // a short unit goes whole to the run that it starts in
    const bool uncut = q.pages <= kWhole;
    if (uncut && u0 < x0) {
      x = u1;
      continue;
    }
    const int begin = (int)(max(x0, u0) - u0), end = uncut ? q.pages : (int)(min(x1, u1) - u0);  // the run's part of it
    const int p0 = (int)(x - u0), p1 = min(end, p0 + kSpan);
    const int R = q.n * G;
    const int32_t* table = a.block_table + (long long)b * a.max_blocks;

    if (used) __syncthreads();  // the last unit's outputs have left shared memory
    used = true;
    // the queries, zeros in place of rows past the last: in the first group of copies
    for (int i = tid; i < kRows * CH; i += kThreads) {
      const int r = i / CH, c = i % CH;
      const long long at = r < R ? (long long)(start + r / G) * a.q_stride + (long long)(kvh * G + r % G) * HD + c * 8 : 0;
      copy16(smem_addr(sQ) + chunk_at<HD>(r, c), static_cast<const bf16*>(a.q) + at, r < R);
    }

    const int last = q.P + q.n - 1;
    const int steps = (p1 - p0 - warp + kWarps - 1) / kWarps;  // pages of this warp; may be 0 or less
    int ids = 0;
    auto ids_from = [&](int k) {  // block of this warp's page k + lane
      const int page = p0 + warp + (k + lane) * kWarps;
      ids = page < p1 ? table[q.position(page) / 16] : 0;
    };
    auto issue = [&](int k) {
      if (k < steps) {
        if (k % 32 == 0) ids_from(k);
        const int blk = __shfl_sync(0xffffffffu, ids, k % 32);
        const int at = q.position(p0 + warp + k * kWarps);
        const long long row0 = ((long long)blk * a.Hkv + kvh) * 16;
        const bf16* ks = static_cast<const bf16*>(a.k_cache) + row0 * HD;
        const bf16* vs = static_cast<const bf16*>(a.v_cache) + row0 * HD;
        const uint32_t dst = my_ring + (k % S::kStages) * 2 * S::kPage;
#pragma unroll
        for (int i = 0; i < CH / 2; ++i) {
          const int r = (i * 32 + lane) / CH, c = (i * 32 + lane) % CH;
          const int j = at + r;
          const bool real = j <= last && (j >= q.lo || j < q.s);
          copy16(dst + chunk_at<HD>(r, c), ks + r * HD + c * 8, real);
          copy16(dst + S::kPage + chunk_at<HD>(r, c), vs + r * HD + c * 8, real);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < S::kStages - 1; ++k) issue(k);
    cp_async_wait<S::kStages - 2>();
    __syncthreads();

    // a thread's rows are lane / 4 and lane / 4 + 8
    int pos[2];
    float m[2], l[2], o[HD / 8][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      pos[h] = q.P + min((lane / 4 + 8 * h) / G, q.n - 1);
      m[h] = -INFINITY, l[h] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < HD / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    constexpr bool kHeld = HD <= 128;  // queries stay in registers
    uint32_t qr[kHeld ? HD / 16 : 1][4];
    const uint32_t q_addr = smem_addr(sQ);
    if constexpr (kHeld) {
#pragma unroll
      for (int c = 0; c < HD / 16; ++c) ldsm4(q_addr + chunk_at<HD>(lane % 16, 2 * c + lane / 16), qr[c]);
    }

    for (int k = 0; k < steps; ++k) {
      issue(k + S::kStages - 1);
      cp_async_wait<S::kStages - 1>();
      __syncwarp();
      const uint32_t kp = my_ring + (k % S::kStages) * 2 * S::kPage, vp = kp + S::kPage;
      float s[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
      for (int c = 0; c < HD / 16; ++c) {
        uint32_t kf[4], qf[4];
        ldsm4(kp + chunk_at<HD>(lane % 8 + (lane / 16) * 8, 2 * c + (lane / 8) % 2), kf);
        if constexpr (kHeld) {
          qf[0] = qr[c][0], qf[1] = qr[c][1], qf[2] = qr[c][2], qf[3] = qr[c][3];
        } else {
          ldsm4(q_addr + chunk_at<HD>(lane % 16, 2 * c + lane / 16), qf);
        }
        mma16816(s[0], qf, kf[0], kf[1]);
        mma16816(s[1], qf, kf[2], kf[3]);
      }
      const int at = q.position(p0 + warp + k * kWarps);
      // every row sees the whole page: up to the first token, and within the last one's window or among the first tokens
      const bool open = at + 15 <= q.P && (a.window == 0 || at > last - a.window || at + 15 < a.sinks);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = s[i][e] * scale;
          if (!open) {
            const int j = at + i * 8 + (lane % 4) * 2 + (e & 1), p = pos[e / 2];
            if (j > p || (a.window > 0 && p - j >= a.window && j >= a.sinks)) v = -INFINITY;
          }
          s[i][e] = v;
        }
      float mx[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mx[h] = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
      }
      if (__any_sync(0xffffffffu, mx[0] > m[0] + kRaise || mx[1] > m[1] + kRaise)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float to = fmaxf(m[h], mx[h]);
          const float f = m[h] == -INFINITY ? 0.f : ex2(m[h] - to);
          m[h] = to;
          l[h] *= f;
#pragma unroll
          for (int i = 0; i < HD / 8; ++i) o[i][2 * h] *= f, o[i][2 * h + 1] *= f;
        }
      }
      uint32_t pf[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float neg = m[h] == -INFINITY ? 0.f : -m[h];  // nothing seen yet: 2^-inf = 0
        pf[h] = pack_bf16x2(ex2(s[0][2 * h] + neg), ex2(s[0][2 * h + 1] + neg));
        pf[2 + h] = pack_bf16x2(ex2(s[1][2 * h] + neg), ex2(s[1][2 * h + 1] + neg));
        // The sum of what the product with the values will use: nearer than that of the fp32 weights where few keys carry a
        // row (scores of sigma 4: outputs off by 0.0018 of their norm in place of 0.0019), and no slower.
        l[h] += (bf16lo(pf[h]) + bf16hi(pf[h])) + (bf16lo(pf[2 + h]) + bf16hi(pf[2 + h]));
      }
#pragma unroll
      for (int c = 0; c < CH; c += 2) {
        uint32_t vf[4];
        ldsm4_t(vp + chunk_at<HD>(lane % 16, c + lane / 16), vf);
        mma16816(o[c], pf, vf[0], vf[1]);
        mma16816(o[c + 1], pf, vf[2], vf[3]);
      }
      __syncwarp();  // the stage is free
    }
    cp_async_wait<0>();

    // The four warps' outputs meet in shared memory, over the rings.
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    __syncthreads();
    float* acc = reinterpret_cast<float*>(ring);  // [kWarps][16][HD]
    float* ml = reinterpret_cast<float*>(sQ);     // [kWarps][16][2]
    static_assert(kWarps * kRows * HD * 4 <= S::kRing, "outputs fit over the rings");
    static_assert(kWarps * 2 * 4 <= HD * 2, "maxima and sums fit over the queries");
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = lane / 4 + 8 * h;
      if (r < R) {
        float* row = acc + (warp * kRows + r) * HD;
#pragma unroll
        for (int i = 0; i < HD / 8; ++i)
          *reinterpret_cast<float2*>(row + i * 8 + (lane % 4) * 2) = make_float2(o[i][2 * h], o[i][2 * h + 1]);
        if (lane % 4 == 0) ml[(warp * kRows + r) * 2] = m[h], ml[(warp * kRows + r) * 2 + 1] = l[h];
      }
    }
    __syncthreads();
    const bool alone = begin == 0 && end == q.pages;
    const long long c0 = quotient(u0, per), c1 = quotient(u1 - 1, per);  // the CTAs that share the unit
    // a CTA's first unit goes to its slot 0, a later one that runs past its end to slot 1, others' parts before that one too
    auto slot_of = [&](long long c) { return slots + (2 * c + (c * per < u0 ? 1 : 0)) * kSlot; };
    auto put = [&](int r, int c, const float* v) {
      uint2 w = pack4(v);
      *reinterpret_cast<uint2*>(static_cast<bf16*>(a.out) + (long long)(start + r / G) * a.out_stride +
                                (long long)(kvh * G + r % G) * HD + c) = w;
    };
    const int after = (end - p1 + kSpan - 1) / kSpan;  // parts to come; the last one's maxima and sums are the first copy
    for (int i = tid; i < R * (HD / 4); i += kThreads) {
      const int r = i / (HD / 4), c = i % (HD / 4) * 4;
      float* slot = slot_of(blockIdx.x);
      float* slot_ml = slot + kRows * HD + r * 2;
      float top = -INFINITY, f[kWarps], sum = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[(w * kRows + r) * 2]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = ml[(w * kRows + r) * 2];
        f[w] = mw == -INFINITY ? 0.f : ex2(mw - top);
        sum += f[w] * ml[(w * kRows + r) * 2 + 1];
        const float4 y = *reinterpret_cast<const float4*>(acc + (w * kRows + r) * HD + c);
        v[0] += f[w] * y.x, v[1] += f[w] * y.y, v[2] += f[w] * y.z, v[3] += f[w] * y.w;
      }
      if (p0 > begin) {  // with the parts before it
        const float2 w = *reinterpret_cast<const float2*>(slot_ml + ((after + 1) & 1) * 2 * kRows);
        const float4 y = *reinterpret_cast<const float4*>(slot + r * HD + c);
        const float to = fmaxf(top, w.x);
        const float f0 = top == -INFINITY ? 0.f : ex2(top - to), f1 = w.x == -INFINITY ? 0.f : ex2(w.x - to);
        top = to;
        sum = f0 * sum + f1 * w.y;
        v[0] = f0 * v[0] + f1 * y.x, v[1] = f0 * v[1] + f1 * y.y;
        v[2] = f0 * v[2] + f1 * y.z, v[3] = f0 * v[3] + f1 * y.w;
      }
      if (alone && after == 0) {
        const float inv = 1.f / sum;
        v[0] *= inv, v[1] *= inv, v[2] *= inv, v[3] *= inv;
        put(r, c, v);
      } else {
        *reinterpret_cast<float4*>(slot + r * HD + c) = make_float4(v[0], v[1], v[2], v[3]);
        if (c == 0) *reinterpret_cast<float2*>(slot_ml + (after & 1) * 2 * kRows) = make_float2(top, sum);
      }
    }
    if (!alone && after == 0) {
      __syncthreads();
      if (tid == 0) {
        __threadfence();
        s_last = atomicAdd(arrived + (long long)b * a.Hkv + kvh, 1) == (int)(c1 - c0);
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        // twelve parts at a time: their loads do not wait for one another
        constexpr int kBatch = 12;
        const int parts = (int)(c1 - c0) + 1;
        for (int i = tid; i < R * (HD / 4); i += kThreads) {
          const int r = i / (HD / 4), c = i % (HD / 4) * 4;
          float top = -INFINITY, sum = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
          for (int k = 0; k < parts; k += kBatch) {
            float2 w[kBatch];
            float4 y[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
              const float* slot = slot_of(c0 + min(k + j, parts - 1));
              w[j] = __ldcg(reinterpret_cast<const float2*>(slot + kRows * HD + r * 2));
              y[j] = __ldcg(reinterpret_cast<const float4*>(slot + r * HD + c));
            }
            float to = top;
#pragma unroll
            for (int j = 0; j < kBatch; ++j) to = fmaxf(to, w[j].x);
            const float f0 = top == -INFINITY ? 0.f : ex2(top - to);
            top = to;
            sum *= f0, v[0] *= f0, v[1] *= f0, v[2] *= f0, v[3] *= f0;
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
              const float f = k + j >= parts || w[j].x == -INFINITY ? 0.f : ex2(w[j].x - to);
              sum += f * w[j].y;
              v[0] += f * y[j].x, v[1] += f * y[j].y, v[2] += f * y[j].z, v[3] += f * y[j].w;
            }
          }
          const float inv = 1.f / sum;
          v[0] *= inv, v[1] *= inv, v[2] *= inv, v[3] *= inv;
          put(r, c, v);
        }
      }
    }
    x = u0 + p1;
  }
}

template <int HD>
cudaError_t go(const WinAttnArgs& a, const long long* cost, int* arrived, float* slots, cudaStream_t s) {
  const size_t smem = kRows * HD * 2 + Shape<HD>::kRing;
  auto kern = window_rows_kernel<HD>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_behind_plan(kern, kSms * per_sm(HD), kThreads, smem, s, a, cost, slots, arrived);
}

}  // namespace

size_t window_rows_slots(int hd) { return (size_t)kSms * per_sm(hd) * 2 * kRows * (hd + 4) * sizeof(float); }

cudaError_t launch_window_rows(const WinAttnArgs& a, const long long* cost, int* arrived, float* slots, cudaStream_t s) {
  if (a.hd == 64) return go<64>(a, cost, arrived, slots, s);
  return a.hd == 128 ? go<128>(a, cost, arrived, slots, s) : go<256>(a, cost, arrived, slots, s);
}

}  // namespace tv
