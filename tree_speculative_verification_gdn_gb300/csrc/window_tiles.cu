// Windowed attention of many query rows -- prompts -- on the 5th-generation tensor cores.
//
// A unit is a run of new tokens of one sequence for one KV head; its query rows, (token, query head of the group), fill
// tiles of 128: two of head dims 64 and 128, one of 256.  Every unit walks its visible pages alone, sixteen tokens each,
// hidden pages between the first tokens and the window left out, 64 keys at a time.  Units of all sequences and KV heads lie
// one behind the other, each as long as its key tiles and kUnitCost more, and a persistent grid takes equal runs of that, so
// that ragged and causal work ends together; a long unit cut by a run's end leaves maximum, sum and unnormalised output per
// row in the workspace, and the last of its CTAs joins them in the order of the runs.
//
// Scores S = Q K^T go to tensor memory, two buffers a row tile; a thread takes a row (TMEM lane) of 64 to registers, and
// 2^(S scale - m) goes back as bf16, to a buffer that O += P V reads.  MMAs with different accumulators need not run in
// order, so nothing is written before the reader of what was there has ended.  Weights in fp32 would be a second product.  The
// sum is of the fp32 weights before their rounding; a sum of the rounded ones is nearer where few keys carry a row (scores of
// sigma 4: outputs off by 0.0019 of their norm in place of 0.0021, the store alone 0.0017; sigma 1: 0.0023 both), but took
// 1.64 ms for 16384 tokens at head dim 128 in place of 1.51.
//   warps 0-3, 4-7   softmax of row tile 0 and 1, output of each (one row tile: two buffers in turn, warps 0-3)
//   warp 8           TMA: queries, K and V tiles through a ring each
//   warp 9, 11       MMAs of scores, of outputs: one warp for both spent longer on its waits and commits than the MMAs took
//   warp 10          the run's units, up to four ahead
//
// Bound by the matrix units and by tensor memory, which they share with the loads and stores of scores and weights.  16384
// tokens, 32 query heads on 8: head dim 64 1.34 ms, 128 1.51 ms (1.46 PFLOP/s), 256 2.82 ms (1.56 PFLOP/s).  The same copies and
// MMAs without the softmax take 1.14, 1.30 and 2.65 ms; without its arithmetic, but with its loads and stores, 1.29, 1.55
// and 2.80.  Tiles of 96 keys, fewer and longer MMAs with one buffer of weights, took 1.40 and 1.57 ms (64, 128); tiles of
// 128, scores and weights in one buffer and a wait between, 1.49 and 1.70.
//
// Values that no token of the unit sees may be anything, and 0 times that is not 0: their rows are cleared in
// shared memory before P V.  Every wait is bounded; a role that gives up makes all leave.
#include "tv_tma_host.h"
#include "tv_tc.cuh"
#include "window_attn.cuh"

namespace tv {
namespace {

constexpr int kRows = 128;
constexpr int kThreads = 384;
constexpr int kUnits = 4;       // units known ahead
// Key tiles of a unit that is never cut: a cut costs about as much.  8 prompts of 500 tokens on the average, window 1024, head dim
// 256: 96 us with 8 for the limit, 84 with 20; 900 tokens alone 46 and 34; two or three units a CTA: up to 5 % the other way.
constexpr int kWhole = 20;
constexpr int kLeast = kUnitCost + 1;  // cost of a run, at least: no two units begin in a shorter one
// Key tiles of a part: the run's share of a unit comes to the roles in parts, whose outputs are joined in the run's slot of
// the workspace.  The matrix units cut what they add to an output, which leaves a sum over n keys short by about n 2^-27.4
// of it: 6e-3 with 2^20, 2.5e-2 with 2^22.  Parts of 2^15, joined in fp32, lose 2e-4, a tenth of the store's rounding; one
// takes some 400 us, its start and output 4.
constexpr int kPart = 512;
constexpr float kRaise = 8.0f;     // log2

template <int HD>
struct Shape {
  static constexpr int NT = HD == 256 ? 1 : 2;          // row tiles
  static constexpr int KT = 64;                         // keys of a tile
  static constexpr int KS = HD == 64 ? 8 : HD == 128 ? 6 : 3;  // K tiles in their ring
  static constexpr int VS = HD == 64 ? 8 : HD == 128 ? 4 : 2;  // V tiles in theirs
  static constexpr uint32_t QCHUNK = kRows * 128;       // 64 columns of a row tile
  static constexpr uint32_t QTILE = HD / 64 * QCHUNK;
  static constexpr uint32_t EIGHT = HD * 16;            // eight keys: 1024 bytes for each 64 of their columns
  static constexpr uint32_t STAGE = KT / 8 * EIGHT;
  static constexpr uint32_t K0 = NT * QTILE;
  static constexpr uint32_t V0 = K0 + KS * STAGE;
  static constexpr uint32_t BARS = V0 + VS * STAGE;
  static constexpr uint32_t TOTAL = BARS + 1024;
  // TMEM: outputs, two buffers of scores a row tile, and as many of weights; head dim 128 leaves no columns for those, and
  // weights lie where their scores were.
  static constexpr bool OVER = HD == 128;
  static constexpr uint32_t S0 = NT * HD, P0 = OVER ? S0 : S0 + NT * 2 * KT, PSTEP = OVER ? KT : KT / 2;
  static constexpr int SLOT = NT * kRows * (HD + 2);    // floats of a cut unit
  static_assert(P0 + NT * 2 * PSTEP <= 512, "tensor memory");
  static_assert(TOTAL + 1024 <= 232448, "shared memory");
};

// A phase of the barrier, or false after 4 s at most, or once another role has given up.  Looks once, then tries, each try
// asleep in the barrier unit for 4 us at most (whatever the hint; measured).  No wait outlasts a part by much, 0.4 ms.
constexpr uint32_t kTries = 1u << 20;
__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile int* abort) {
  for (uint32_t it = 0; it < kTries; ++it) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity), "r"(1000u)
        : "memory");
    if (done) return true;
    if (*abort) return false;
  }
  *abort = 1;
  return false;
}
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return mbar_test(bar, parity) || wait_long(bar, parity, abort);
}

// The MMA warp runs as one, so that addresses stay in uniform registers; one elected lane issues.
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}
// Shared-memory descriptors of 128-byte swizzled operands, in two words: the start and the bytes from 64 columns to the
// next 64 (operands with the columns outermost), and the bytes from eight rows to the next eight.
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t columns) {
  return (saddr >> 4) | (columns >> 4) << 16;
}
__host__ __device__ constexpr uint32_t desc_high(uint32_t eight_rows) { return (eight_rows >> 4) | (1u << 14) | (2u << 29); }
template <uint32_t A_HIGH, uint32_t B_HIGH>
__device__ __forceinline__ void mma_ss(uint32_t elected, uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 a, {%1, %6};\n\tmov.b64 b, {%2, %7};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(a_low), "r"(b_low), "r"(idesc), "r"(accumulate), "r"(elected), "n"(A_HIGH), "n"(B_HIGH)
      : "memory");
}
template <uint32_t B_HIGH>
__device__ __forceinline__ void mma_ts(uint32_t elected, uint32_t d, uint32_t a_tmem, uint32_t b_low, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 b, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_low), "r"(idesc), "r"(accumulate), "r"(elected), "n"(B_HIGH)
      : "memory");
}
// One arrival of a warp.
__device__ __forceinline__ void arrive_of(int lane, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.eq.s32 q, %1, 0;\n\t"
      "@q mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_addr(bar)),
      "r"(lane)
      : "memory");
}
__device__ __forceinline__ void commit_to(uint32_t elected, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)),
      "r"(elected)
      : "memory");
}

__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// until loads have landed; r is theirs, and not used before
__device__ __forceinline__ void tmem_landed(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :: "memory");
  asm volatile(""
               : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :: "memory");
}
__device__ __forceinline__ void tmem_landed(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :: "memory");
}
__device__ __forceinline__ void tmem_st16_nowait(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A unit, or a part of its key tiles that lie in the CTA's run.
struct Unit {
  int more;                // 0: the run has ended
  int b, kvh, token;       // sequence, KV head, first token's row
  int tiles, begin, end;   // key tiles of the unit, the run's share of them
  int first, last;         // the part's
  int c0, c1;              // the CTAs that share it
  Seen seen;
};

struct Bars {
  uint64_t q_full, q_free;
  uint64_t k_full[8], k_empty[8], v_full[8], v_empty[8];
  uint64_t s_full[4], s_read[4], p_full[4], pv_done[4], o_free[2];
  uint64_t unit_full[kUnits], unit_empty[kUnits];
  uint64_t drain;
  uint32_t tmem;
  int abort;
  Unit units[kUnits];
};
static_assert(sizeof(Bars) <= 1024, "barriers fit their region");

// The units of a run, in order.  Made by a whole warp, walked by any thread of it.
struct Walk {
  const WinAttnArgs& a;
  const long long* cost;
  const Run& run;
  TileShape shape;
  int t, start, n, P;  // first token of the unit in the sequence; the sequence
  long long u0;        // where the unit's cost starts
  Unit u;

  __device__ void sequence() {
    start = a.cu != nullptr ? a.cu[u.b] : u.b;
    n = a.cu != nullptr ? a.cu[u.b + 1] - start : 1;
    P = a.prefix_len[u.b];
    t = 0;
  }
  __device__ int tiles_of(int first_token) const {
    return (seen_by(a, P + first_token, min(shape.tokens, n - first_token)).pages * 16 + shape.keys - 1) / shape.keys;
  }
  __device__ void unit() {
    u.seen = seen_by(a, P + t, min(shape.tokens, n - t));
    u.token = start + t;
    u.tiles = (u.seen.pages * 16 + shape.keys - 1) / shape.keys;
    if (u.tiles <= kWhole) {  // to the run that it starts in
      u.begin = 0, u.end = u0 >= run.x0 && u0 < run.x1 ? u.tiles : 0;
    } else {
      const long long k0 = u0 + kUnitCost;
      u.begin = (int)min((long long)u.tiles, max(0LL, run.x0 - k0));
      u.end = (int)max(0LL, min((long long)u.tiles, run.x1 - k0));
    }
  }
  __device__ void part(int first) { u.first = first, u.last = min(u.end, first + kPart); }
  __device__ Walk(const WinAttnArgs& a_, const long long* cost_, const Run& run_, TileShape s)
      : a(a_), cost(cost_), run(run_), shape(s) {
    u.b = run.b;
    start = run.start, n = run.n, P = run.P, t = 0;
    const long long c = cost[u.b];
    u.kvh = (int)quotient(run.x0 - run.base, c);
    u0 = run.base + u.kvh * c;
    // a unit a lane, 32 at a time
    for (;;) {
      const int lane = threadIdx.x % 32;
      const long long t_lane = t + (long long)lane * shape.tokens;
      int upto = t_lane < n ? kUnitCost + tiles_of((int)t_lane) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const unsigned past = __ballot_sync(0xffffffffu, u0 + upto > run.x0);
      const int skip = past != 0 ? __ffs(past) - 1 : 32;
      if (skip > 0) u0 += __shfl_sync(0xffffffffu, upto, skip - 1);
      t += skip * shape.tokens;
      if (past != 0) break;
    }
    unit();
    settle();
  }
  // On from a unit that has no key tile in the run.
  __device__ void settle() {
    while (u0 < run.x1 && u.begin >= u.end) step();
    u.more = u0 < run.x1;
    part(u.begin);
    const long long k0 = u0 + kUnitCost;
    u.c0 = (int)quotient(k0, run.per), u.c1 = (int)quotient(k0 + u.tiles - 1, run.per);
  }
  __device__ void step() {
    u0 += kUnitCost + u.tiles;
    if (u0 >= run.x1) return;
    t += shape.tokens;
    if (t >= n) {
      t = 0;
      if (++u.kvh == a.Hkv) {
        u.kvh = 0;
        while (cost[++u.b] == 0) {}
        sequence();
      }
    }
    unit();
  }
  __device__ void next() {
    if (u.last < u.end) return part(u.last);
    step();
    settle();
  }
};

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    window_tiles_kernel(const __grid_constant__ WinAttnArgs a, const long long* cost, int* arrived, float* slots, int npt,
                        const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                        const __grid_constant__ CUtensorMap mV) {
  using L = Shape<HD>;
  constexpr int NT = L::NT, KT = L::KT, KS = L::KS, VS = L::VS;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  unsigned char* sm = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  Bars& bar = *reinterpret_cast<Bars*>(sm + L::BARS);
  volatile int* abort = &bar.abort;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int G = a.Hq / a.Hkv;

  if (tid == 0) {
    mbar_init(&bar.q_full, 1);
    mbar_init(&bar.q_free, 1);
    for (int s = 0; s < KS; ++s) {
      mbar_init(&bar.k_full[s], 1);
      mbar_init(&bar.k_empty[s], 1);
    }
    for (int s = 0; s < VS; ++s) {
      mbar_init(&bar.v_full[s], 1);
      mbar_init(&bar.v_empty[s], 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&bar.s_full[s], 1);
      mbar_init(&bar.s_read[s], 4);
      mbar_init(&bar.p_full[s], 4);
      mbar_init(&bar.pv_done[s], 1);
    }
    mbar_init(&bar.o_free[0], 4);
    mbar_init(&bar.o_free[1], 4);
    for (int s = 0; s < kUnits; ++s) {
      mbar_init(&bar.unit_full[s], 1);
      mbar_init(&bar.unit_empty[s], 11);
    }
    mbar_init(&bar.drain, 2);
    bar.abort = 0;
    mbar_fence_init();
  }
  if (warp == 9) tmem_alloc(&bar.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;
  wait_for_plan();
  Run run;
  if (!find_run<kThreads>(a, cost, kLeast, run)) {
    __syncthreads();
    if (warp == 9) tmem_dealloc(tmem, 512);
    return;
  }
  uint32_t k_loads = 0, v_loads = 0, q_loads = 0;  // what the producer has started
  // the k-th unit, once it is known; a warp hands it back when it needs no more of it
  auto known = [&](uint32_t k) -> bool {
    return __all_sync(0xffffffffu, wait_for(&bar.unit_full[k % kUnits], k / kUnits & 1, abort));
  };
  auto hand_back = [&](uint32_t k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar.unit_empty[k % kUnits]);
  };

  auto advance = [](uint32_t& st, uint32_t& ph, uint32_t stages) {
    if (++st == stages) st = 0, ph ^= 1;
  };

  if (warp == 10) {
    // ---------------------------------------------------------------- units
    Walk w(a, cost, run, TileShape{NT * npt, KT});
    if (lane == 0) {
      for (uint32_t k = 0;; ++k) {
        if (k >= kUnits && !wait_for(&bar.unit_empty[k % kUnits], (k / kUnits - 1) & 1, abort)) break;
        bar.units[k % kUnits] = w.u;
        mbar_arrive(&bar.unit_full[k % kUnits]);
        if (!w.u.more) break;
        w.next();
      }
    }
  } else if (warp == 8) {
    // ---------------------------------------------------------------- TMA (whole warp; lane p has page p of a tile)
    constexpr int PAGES = KT / 16;
    bool ok = true;
    for (uint32_t unit = 0; ok && known(unit); hand_back(unit), ++unit) {
      const Unit w = bar.units[unit % kUnits];
      if (!w.more) break;
      const int32_t* table = a.block_table + (long long)w.b * a.max_blocks;
      auto block_of = [&](int tile) {  // pages past the last are that one again: their columns are masked
        const int page = min(tile * PAGES + lane, w.seen.pages - 1);
        return lane < PAGES && tile < w.last ? table[w.seen.position(page) / 16] : 0;
      };
      auto load = [&](const CUtensorMap* map, uint32_t ring, uint32_t stages, uint64_t* fulls, uint64_t* empties, uint32_t& loads,
                      int blk) -> bool {
        const uint32_t st = loads % stages;
        if (loads >= stages && !__all_sync(0xffffffffu, wait_for(&empties[st], (loads / stages - 1) & 1, abort))) return false;
        if (lane == 0) mbar_arrive_expect_tx(&fulls[st], L::STAGE);
        __syncwarp();
        if (lane < PAGES)
          tma_load_4d(sm + ring + st * L::STAGE + lane * 2 * L::EIGHT, map, 0, 0, 0, (blk * a.Hkv + w.kvh) * 2, &fulls[st]);
        ++loads;
        return true;
      };
      // keys run two tiles ahead of values: scores are made that much earlier than outputs
      int blk[3];
#pragma unroll
      for (int k = 0; k < 3; ++k) blk[k] = block_of(w.first + k);
      ok = load(&mK, L::K0, KS, bar.k_full, bar.k_empty, k_loads, blk[0]);
      if (ok && w.first + 1 < w.last) ok = load(&mK, L::K0, KS, bar.k_full, bar.k_empty, k_loads, blk[1]);
      for (int i = w.first; ok && i < w.last; ++i) {
        const int after = block_of(i + 3);
        if (i + 2 < w.last) ok = load(&mK, L::K0, KS, bar.k_full, bar.k_empty, k_loads, blk[2]);
        if (ok && i == w.first) {  // queries behind the first keys, which need not wait for the last unit's queries
          if (unit > 0) ok = __all_sync(0xffffffffu, wait_for(&bar.q_free, (unit - 1) & 1, abort));
          if (!ok) break;
          const int tiles = NT == 2 && w.seen.n > npt ? 2 : 1;
          if (lane == 0) {
            mbar_arrive_expect_tx(&bar.q_full, tiles * (uint32_t)(HD * G * npt * 2));
            for (int x = 0; x < tiles; ++x)
              for (int c = 0; c < HD / 64; ++c)
                tma_load_4d(sm + x * L::QTILE + c * L::QCHUNK, &mQ, c * 64, 0, w.kvh, w.token + x * npt, &bar.q_full);
          }
          ++q_loads;
        }
        ok = ok && load(&mV, L::V0, VS, bar.v_full, bar.v_empty, v_loads, blk[0]);
        blk[0] = blk[1], blk[1] = blk[2], blk[2] = after;
      }
    }
  } else if (warp == 9) {
    // ---------------------------------------------------------------- scores
    constexpr uint32_t idS = idesc_bf16_f32(128, KT);
    const uint32_t elected = elect_lane();
    const uint32_t q_low = desc_low(smem_addr(sm), 16), k_low = desc_low(smem_addr(sm + L::K0), 16);
    constexpr uint32_t q_high = desc_high(1024), k_high = desc_high(L::EIGHT);
    uint32_t kst = 0, kph = 0;             // stage and phase of the ring
    uint32_t used = 0, free_phase = 0;     // a bit a buffer: whether any scores were made in it; the phase of its being free
    bool ok = true;
    auto wait = [&](uint64_t* w, uint32_t parity) { return __all_sync(0xffffffffu, wait_for(w, parity, abort)); };
    for (uint32_t unit = 0; ok && known(unit); hand_back(unit), ++unit) {
      const Unit& w = bar.units[unit % kUnits];
      if (!w.more) break;
      const bool two = NT == 2 && __shfl_sync(0xffffffffu, w.seen.n, 0) > npt;
      const int tiles = __shfl_sync(0xffffffffu, w.last - w.first, 0);
      ok = wait(&bar.q_full, unit & 1);
      // Scores of row tile x from the keys of the stage into buffer sb, once its scores have been read, and the weights over
      // them too.  A waiter has to see every phase of a barrier, none of them two late: each barrier here is for one buffer.
      auto scores = [&](int x, int sb) -> bool {
        if (used >> sb & 1) {
          if (!wait(L::OVER ? &bar.pv_done[sb] : &bar.s_read[sb], free_phase >> sb & 1)) return false;
          free_phase ^= 1u << sb;
        }
        used |= 1u << sb;
        tc_fence_after();
        const uint32_t q = q_low + x * (L::QTILE >> 4), k = k_low + kst * (L::STAGE >> 4), d = tmem + L::S0 + sb * KT;
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          mma_ss<q_high, k_high>(elected, d, q + ((kk / 4 * L::QCHUNK + kk % 4 * 32) >> 4),
                                 k + ((kk / 4 * 1024 + kk % 4 * 32) >> 4), idS, kk ? 1u : 0u);
        commit_to(elected, &bar.s_full[sb]);
        return true;
      };
      for (int j = 0; ok && j < tiles; ++j) {
        ok = wait(&bar.k_full[kst], kph) && scores(0, j & 1) && (!two || scores(1, 2 + (j & 1)));
        commit_to(elected, &bar.k_empty[kst]);
        advance(kst, kph, KS);
      }
      commit_to(elected, &bar.q_free);
    }
  } else if (warp == 11) {
    // ---------------------------------------------------------------- outputs
    constexpr uint32_t idO = idesc_bf16_f32(128, HD, true);
    const uint32_t elected = elect_lane();
    const uint32_t v_low = desc_low(smem_addr(sm + L::V0), 1024);
    constexpr uint32_t v_high = desc_high(L::EIGHT);
    uint32_t vst = 0, vph = 0;             // stage and phase of the ring
    uint32_t p_phase = 0, units[2] = {0, 0};  // p_phase: a bit a buffer of weights
    bool ok = true;
    auto wait = [&](uint64_t* w, uint32_t parity) { return __all_sync(0xffffffffu, wait_for(w, parity, abort)); };
    for (uint32_t unit = 0; ok && known(unit); hand_back(unit), ++unit) {
      const Unit& w = bar.units[unit % kUnits];
      if (!w.more) break;
      const bool two = NT == 2 && __shfl_sync(0xffffffffu, w.seen.n, 0) > npt;
      const int tiles = __shfl_sync(0xffffffffu, w.last - w.first, 0);
      // output of row tile x from the values of the stage and the weights in buffer pb
      auto outputs = [&](int x, int pb, bool fresh) -> bool {
        if (fresh && units[x] > 0 && !wait(&bar.o_free[x], (units[x] - 1) & 1)) return false;
        if (!wait(&bar.p_full[pb], p_phase >> pb & 1)) return false;
        p_phase ^= 1u << pb;
        tc_fence_after();
        const uint32_t v = v_low + vst * (L::STAGE >> 4), p = tmem + L::P0 + pb * L::PSTEP;
#pragma unroll
        for (int kk = 0; kk < KT / 16; ++kk)
          mma_ts<v_high>(elected, tmem + x * HD, p + kk * 8, v + (kk * 2 * L::EIGHT >> 4), idO, (!fresh || kk > 0) ? 1u : 0u);
        commit_to(elected, &bar.pv_done[pb]);
        return true;
      };
      for (int j = 0; ok && j < tiles; ++j) {
        ok = wait(&bar.v_full[vst], vph) && outputs(0, j & 1, j == 0) && (!two || outputs(1, 2 + (j & 1), j == 0));
        commit_to(elected, &bar.v_empty[vst]);
        advance(vst, vph, VS);
      }
      ++units[0];
      if (two) ++units[1];
    }
  } else if (warp < 8) {
    // ---------------------------------------------------------------- softmax and output, a row a thread
    const int wg = warp / 4;                 // row tile
    const int r = tid % kRows, i_row = r / G, g = r % G;
    const uint32_t lanes = (uint32_t)(32 * (warp % 4)) << 16;
    const float sign = a.sm_scale < 0.f ? -1.f : 1.f;
    // a scale of 0 has to leave hidden keys at -inf: the smallest number serves
    const float scale = fmaxf(fabsf(a.sm_scale) * 1.4426950408889634f, 1.17549435e-38f);
    uint32_t s_phase = 0, seq = 0;          // s_phase: a bit a barrier of scores
    uint32_t weighed = 0, pv_phase = 0;     // a bit a buffer of weights: outputs from it not seen to be over; their phase
    bool ok = true;
    // until the outputs from this row tile's buffer b of weights are over; `over`: what a look at the barrier said
    auto look = [&](int b) -> bool { return !(weighed >> b & 1) || mbar_test(&bar.pv_done[2 * wg + b], pv_phase >> b & 1); };
    auto outputs_over = [&](int b, bool over) -> bool {
      if (!__all_sync(0xffffffffu, over) &&
          !__all_sync(0xffffffffu, wait_long(&bar.pv_done[2 * wg + b], pv_phase >> b & 1, abort)))
        return false;
      pv_phase ^= weighed & 1u << b, weighed &= ~(1u << b);
      return true;
    };
    for (uint32_t unit = 0; ok && known(unit); hand_back(unit), ++unit) {
      const Unit& w = bar.units[unit % kUnits];
      if (!w.more) break;
      const bool two = NT == 2 && w.seen.n > npt;
      const int tiles = w.last - w.first;
      if (wg == 0 || two) {
        const Seen& q = w.seen;
        const int token = wg * npt + i_row;  // in the unit
        const bool active = i_row < npt && token < q.n;
        // Columns, numbered by visible pages: [0, vs) and [va, ve) are this row's; [h0, h1) and from `end` on no row's.
        int vs = 0, va = 0, ve = 0;
        const int shift = (q.front - q.from) * 16, end = q.P + q.n + shift, h0 = q.s, h1 = q.lo + shift;
        if (active) {
          const int pos = q.P + token;
          ve = pos + 1 + shift;
          va = (a.window > 0 ? max(0, pos - a.window + 1) : 0) + shift;
          vs = min(a.sinks, q.front > 0 ? q.front * 16 : ve);
          if (q.from > 0 && q.front == 0) vs = 0;
        }
        // the columns that every row of the warp sees; rows of no token do not count, here and below
        const int all_vs = __reduce_min_sync(0xffffffffu, active ? vs : 0x7fffffff),
                  all_va = __reduce_max_sync(0xffffffffu, active ? va : 0),
                  all_ve = __reduce_min_sync(0xffffffffu, active ? ve : 0x7fffffff);
        float m = -INFINITY, l = 0.f;
        int c0 = w.first * KT;
        auto look_at_scores = [&](int j) -> bool {
          const int sb = 2 * wg + (j & 1);
          return mbar_test(&bar.s_full[sb], s_phase >> sb & 1);
        };
        bool there = look_at_scores(0);
        for (int j = 0; j < tiles; ++j, c0 += KT) {
          // Each look at a barrier is made a while before its answer is needed: it takes some hundred cycles.
          const int sb = 2 * wg + (j & 1);
          if (!__all_sync(0xffffffffu, there) &&
              !(ok = __all_sync(0xffffffffu, wait_long(&bar.s_full[sb], s_phase >> sb & 1, abort))))
            break;
          s_phase ^= 1u << sb;
          tc_fence_after();
          // the scores to registers, and their buffer back
          uint32_t s0[32], s1[32];
          tmem_ld32_nowait(tmem + L::S0 + sb * KT + lanes, s0);
          tmem_ld32_nowait(tmem + L::S0 + sb * KT + lanes + 32, s1);
          const bool over = L::OVER || look(j & 1);  // OVER: the scores were not made before
          tmem_landed(s0);
          tmem_landed(s1);
          tc_fence_before();
          __syncwarp();
          if (!L::OVER) arrive_of(lane, &bar.s_read[sb]);
          if (sign < 0.f || !((c0 >= all_va && c0 + KT <= all_ve) || c0 + KT <= all_vs)) {
            // hidden keys to -inf
            auto below = [](int n) -> uint32_t { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; };
            const uint32_t b0 = below(vs - c0) | (below(ve - c0) & ~below(va - c0));
            const uint32_t b1 = below(vs - c0 - 32) | (below(ve - c0 - 32) & ~below(va - c0 - 32));
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              s0[k] = (b0 >> k) & 1u ? __float_as_uint(__uint_as_float(s0[k]) * sign) : 0xff800000u;
              s1[k] = (b1 >> k) & 1u ? __float_as_uint(__uint_as_float(s1[k]) * sign) : 0xff800000u;
            }
          }
          // the weights that lay in their place have been read
          ok = outputs_over(j & 1, over);
          if (!ok) break;
          const uint32_t tp = tmem + L::P0 + sb * L::PSTEP + lanes;
          if (wg == 0 && ((h0 < h1 && h0 < c0 + KT && h1 > c0) || end < c0 + KT)) {
            const uint32_t vq = seq + j, vst = vq % VS;
            ok = __all_sync(0xffffffffu, wait_for(&bar.v_full[vst], vq / VS & 1, abort));
            if (!ok) break;
            unsigned char* v = sm + L::V0 + vst * L::STAGE;
#pragma unroll 1
            for (int row = r / 8; row < KT; row += 16) {
              const int c = c0 + row;
              if ((c >= h0 && c < h1) || c >= end)
#pragma unroll
                for (int k = 0; k < HD / 64; ++k)
                  *reinterpret_cast<uint4*>(v + row / 8 * L::EIGHT + k * 1024 + row % 8 * 128 + r % 8 * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async();
          }
          // m is the maximum of some earlier keys of the row; it is raised, and O and l scaled to it, when these keys' is
          // larger by more than 2^kRaise, which is rare: weights up to that do no harm in fp32 and bf16.  With the maximum
          // known first, weights take the scores' place in registers.  Weights made first, and again where their sum showed a
          // larger score, kept both: the compiler then waited for each pair, 1030 cycles for 64 of two warps and not 710.
          {
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 32; c += 4)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                top[k] = fmaxf(fmaxf(top[k], __uint_as_float(s0[c + k])), __uint_as_float(s1[c + k]));
            const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale;
            const bool raise = active && mx > m + kRaise;
            if (__any_sync(0xffffffffu, raise)) {
              const bool rescale = raise && m != -INFINITY;
              if (__any_sync(0xffffffffu, rescale)) {
                // O holds earlier keys: their products have to be done before this warp's rows are scaled
                ok = outputs_over(~j & 1, look(~j & 1));
                if (!ok) break;
                tc_fence_after();
                const float f = rescale ? ex2_approx(m - mx) : 1.f;
                l *= f;
#pragma unroll 1
                for (int c = 0; c < HD; c += 16) {
                  uint32_t o[16];
                  tmem_ld16_nowait(tmem + wg * HD + lanes + c, o);
                  tmem_landed(o);
#pragma unroll
                  for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                  tmem_st16_nowait(tmem + wg * HD + lanes + c, o);
                }
                tmem_wait_st();
              }
              if (raise) m = mx;
            }
            // 2^(s scale - m); a row that has seen nothing yet keeps m = -inf, and 2^-inf = 0
            const float neg = m == -INFINITY ? 0.f : -m;
            const float2 scale2 = make_float2(scale, scale), neg2 = make_float2(neg, neg);
            float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
            auto part = [&](const uint32_t* v, uint32_t at) {
              uint32_t p[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float2 e = __ffma2_rn(
                    make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), scale2, neg2);
                const float2 w2 = make_float2(ex2_approx(e.x), ex2_approx(e.y));
                p[k] = pack_bf16x2(w2.x, w2.y);
                if (k & 1) sum1 = __fadd2_rn(sum1, w2);
                else sum0 = __fadd2_rn(sum0, w2);
              }
              tmem_st16_nowait(at, p);
            };
            part(s0, tp);
            part(s1, tp + 16);
            sum0 = __fadd2_rn(sum0, sum1);
            l += sum0.x + sum0.y;
          }
          there = look_at_scores(j + 1);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          arrive_of(lane, &bar.p_full[sb]);
          weighed |= 1u << (j & 1);
        }
        ok = ok && outputs_over(0, look(0)) && outputs_over(1, look(1));
        if (ok) {
          tc_fence_after();
          const bool whole = w.end - w.begin == w.tiles, done = w.last == w.end;
          bf16* out = static_cast<bf16*>(a.out) + (long long)(w.token + token) * a.out_stride +
                      (long long)(w.kvh * G + g) * HD;
          const int c0 = w.c0, c1 = w.c1;
          // a unit that ends in a later run lies in its first CTA's slot 1, in the others' slot 0; parts of whole ones before it
          // pass through slot 1
          auto slot_of = [&](int c) { return slots + (long long)(2 * c + (c == c0 ? 1 : 0)) * L::SLOT + warp * 32 * (HD + 2); };
          float* mine = slot_of(blockIdx.x);
          const uint32_t from = tmem + wg * HD + lanes;
          if (w.first > w.begin) {  // with the parts before it
            const float2 ml = *reinterpret_cast<const float2*>(mine + 32 * HD + lane * 2);
            const float top = fmaxf(m, ml.x);
            const float f0 = m == -INFINITY ? 0.f : ex2_approx(m - top), f1 = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - top);
            m = top, l = fmaf(l, f0, ml.y * f1);
#pragma unroll 1
            for (int c = 0; c < HD; c += 16) {
              uint32_t o[16];
              tmem_ld16_nowait(from + c, o);
              tmem_landed(o);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float4 y = *reinterpret_cast<const float4*>(mine + (c / 4 + k) * 128 + lane * 4);
                o[4 * k] = __float_as_uint(fmaf(__uint_as_float(o[4 * k]), f0, y.x * f1));
                o[4 * k + 1] = __float_as_uint(fmaf(__uint_as_float(o[4 * k + 1]), f0, y.y * f1));
                o[4 * k + 2] = __float_as_uint(fmaf(__uint_as_float(o[4 * k + 2]), f0, y.z * f1));
                o[4 * k + 3] = __float_as_uint(fmaf(__uint_as_float(o[4 * k + 3]), f0, y.w * f1));
              }
              tmem_st16_nowait(from + c, o);
            }
            tmem_wait_st();
          }
          const float inv = 1.f / l;
          auto put = [&](const uint32_t* o, int c) {
            if (!whole || !done) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                *reinterpret_cast<uint4*>(mine + (c / 4 + k) * 128 + lane * 4) =
                    make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            } else if (active) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float y[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) y[x] = __uint_as_float(o[8 * k + x]) * inv;
                *reinterpret_cast<uint4*>(out + c + 8 * k) = pack8(y);
              }
            }
          };
          // 32 columns on their way while 32 are stored
          uint32_t o0[32], o1[32];
          tmem_ld32_nowait(from, o0);
#pragma unroll 1
          for (int c = 0; c < HD; c += 64) {
            tmem_landed(o0);
            tmem_ld32_nowait(from + c + 32, o1);
            put(o0, c);
            tmem_landed(o1);
            if (c + 64 < HD) tmem_ld32_nowait(from + c + 64, o0);
            put(o1, c + 32);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.o_free[wg]);
          if (!whole || !done) *reinterpret_cast<float2*>(mine + 32 * HD + lane * 2) = make_float2(m, l);
          if (!whole && done) {
            __threadfence();
            __syncwarp();
            int before = 0;
            if (lane == 0) before = atomicAdd(arrived + c0 * 8 + warp, 1);
            if (__shfl_sync(0xffffffffu, before, 0) == c1 - c0) {
              __threadfence();
              float top = -INFINITY, sum = 0.f;
#pragma unroll 8
              for (int c = c0; c <= c1; ++c) top = fmaxf(top, __ldcg(slot_of(c) + 32 * HD + lane * 2));
#pragma unroll 1
              for (int k = 0; k < HD / 4; k += 8) {  // 32 columns: eight loads at once
                float y[32];
#pragma unroll
                for (int x = 0; x < 32; ++x) y[x] = 0.f;
                sum = 0.f;
#pragma unroll 1
                for (int c = c0; c <= c1; ++c) {
                  const float* slot = slot_of(c);
                  const float2 ml = __ldcg(reinterpret_cast<const float2*>(slot + 32 * HD + lane * 2));
                  float4 u[8];
#pragma unroll
                  for (int x = 0; x < 8; ++x) u[x] = __ldcg(reinterpret_cast<const float4*>(slot + (k + x) * 128 + lane * 4));
                  const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - top);
                  sum += f * ml.y;
#pragma unroll
                  for (int x = 0; x < 8; ++x) {
                    y[4 * x] += f * u[x].x, y[4 * x + 1] += f * u[x].y;
                    y[4 * x + 2] += f * u[x].z, y[4 * x + 3] += f * u[x].w;
                  }
                }
                const float total = 1.f / sum;
#pragma unroll
                for (int x = 0; x < 32; ++x) y[x] *= total;
                if (active)
#pragma unroll
                  for (int x = 0; x < 4; ++x) *reinterpret_cast<uint4*>(out + 4 * k + 8 * x) = pack8(y + 8 * x);
              }
            }
          }
        }
      }
      seq += tiles;
    }
  }
  __syncthreads();
  if (bar.abort) {  // what this CTA started ends before its memory goes away
    if (warp == 9 || warp == 11) {
      commit_to(elect_lane(), &bar.drain);
      mbar_wait(&bar.drain, 0);
    }
    if (warp == 8 && lane == 0) {
      if (q_loads > 0) mbar_wait(&bar.q_full, (q_loads - 1) & 1);
      for (uint32_t k = k_loads > KS ? k_loads - KS : 0; k < k_loads; ++k) mbar_wait(&bar.k_full[k % KS], k / KS & 1);
      for (uint32_t k = v_loads > VS ? v_loads - VS : 0; k < v_loads; ++k) mbar_wait(&bar.v_full[k % VS], k / VS & 1);
    }
    if (tid == 0) {
      long long x = run.base;
      for (int b = run.b; x < run.x1; ++b) {
        if (cost[b] > 0) a.err[b] = TV_ERR_TIMEOUT;
        x += cost[b] * a.Hkv;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

template <int HD>
cudaError_t go(const WinAttnArgs& a, const long long* cost, int* arrived, float* slots, cudaStream_t s) {
  using L = Shape<HD>;
  const int G = a.Hq / a.Hkv, npt = kRows / G;
  CUtensorMap mQ, mK, mV;
  {
    const cuuint64_t dims[4] = {(cuuint64_t)HD, (cuuint64_t)G, (cuuint64_t)a.Hkv, (cuuint64_t)a.T};
    const cuuint64_t strides[3] = {(cuuint64_t)HD * 2, (cuuint64_t)G * HD * 2, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)G, 1, (cuuint32_t)npt};
    if (!make_map_bf16_sw128(&mQ, a.q, 4, dims, strides, box)) return cudaErrorInvalidValue;
  }
  {
    // A page of a head, 16 keys, in one copy: eight keys by eight keys, each 64 columns by 64 columns.  With a copy for
    // each 64 columns the copies' number was the limit: 77 cycles each, 27 bytes a cycle on an SM; 4 KB at a time 38, 8 KB 50.
    const cuuint64_t dims[4] = {64, 8, HD / 64, (cuuint64_t)a.num_blocks * a.Hkv * 2};
    const cuuint64_t strides[3] = {(cuuint64_t)HD * 2, 128, (cuuint64_t)8 * HD * 2};
    const cuuint32_t box[4] = {64, 8, HD / 64, 2};
    if (!make_map_bf16_sw128(&mK, a.k_cache, 4, dims, strides, box)) return cudaErrorInvalidValue;
    if (!make_map_bf16_sw128(&mV, a.v_cache, 4, dims, strides, box)) return cudaErrorInvalidValue;
  }
  const size_t smem = L::TOTAL + 1024;
  auto kern = window_tiles_kernel<HD>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_behind_plan(kern, kSms, kThreads, smem, s, a, cost, arrived, slots, npt, mQ, mK, mV);
}

}  // namespace

TileShape window_tile_shape(int Hq, int Hkv, int hd) {
  const int npt = kRows / (Hq / Hkv);
  return TileShape{hd == 256 ? npt : 2 * npt, 64};
}

size_t window_tiles_slots(int hd) {
  const size_t slot = (size_t)(hd == 256 ? 1 : 2) * kRows * (hd + 2) * sizeof(float);
  return 2 * kSms * slot;
}

cudaError_t launch_window_tiles(const WinAttnArgs& a, const long long* cost, int* arrived, float* slots, cudaStream_t s) {
  if (a.hd == 64) return go<64>(a, cost, arrived, slots, s);
  return a.hd == 128 ? go<128>(a, cost, arrived, slots, s) : go<256>(a, cost, arrived, slots, s);
}

}  // namespace tv
