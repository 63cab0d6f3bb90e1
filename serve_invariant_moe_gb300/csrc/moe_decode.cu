// moe_decode.cu -- the whole MoE layer of at most 16 tokens in one kernel (sm_103a).
//
//   l = x Wr^T;  experts and weights of each token from l;  h_e = bf16(silu(x Wg_e) (x Wu_e));  y_e = h_e Wd_e;
//   out = sum_j weight_j y_j + y_shared
//
// Bound by reading the weights of the experts that some token chose, once.  As a chain of kernels (moe_layer_forward) every
// product ends in a partly filled wave and every launch in a gap; here one persistent, cooperatively launched kernel walks
// one list of units, taken from a counter:
//     router (16 experts), the shared expert's gate/up and down, | gate/up of the chosen experts, down of the chosen experts
// A unit is 64 gate rows (48, 32 or 16 where that spreads them better) with the matching up rows, or 128 (64) rows of a down
// projection, over their whole K; what is behind the bar needs the choice.  Weights stream through a shared-memory ring ahead
// of every dependency: one thread loads weights as soon as a stage is free, another one the tokens' side, and only that one
// waits until h is there.  What blocks wait for are counters in the workspace: the router's units done (then every block
// makes the choice for itself, from the logits, into shared memory), an expert's gate/up units done.  No block waits for a
// unit that the counter has not handed out before its own, and a cooperative launch keeps all blocks resident, so every wait
// ends; each has a time limit all the same.  The block that finishes the last unit of a column of outputs combines it, in
// rank order.
//
// The tensor cores do the products although a unit of 16 tokens keeps them nearly idle: an element's bits are those of the
// other engines (K ascending in K = 16 steps of one accumulation chain, no split), so a token's output here is, bit for bit,
// what moe_layer_forward gives it in any batch.  Weights are the MMA's M side (128 rows; 64 for units of at most 64 and for
// the router, whose chain of K / 16 dependent MMAs is what everything else waits for), the tokens its N side, all 16 columns
// of it: gate/up takes x as it is and keeps the columns of the tokens that chose the expert.
//
// Measured as a graph, weights changing from call to call (the chain of kernels in brackets): 256 experts of 6144 x 2048 and
// a shared one, one token 109 to 110 us for 683 MB, 6.2 TB/s (147); 8 tokens that reach 43 to 50 experts 482 to 552, 6.9 TB/s
// (the chain of kernels about a tenth more).  128 experts of 2048 x 768, one token 29 us for 76 MB (46), 16 tokens 119 (162).
// 8 experts of 256 x 512, one token 15 (25).  Where one token's time goes, by stamps in a call of its own with cold caches: the
// large layer (120 us) has all logits after 14 and the choice after 18, behind which only the shared expert's 75 MB are read;
// its last down unit after 117.  The layer of 128 experts (31 us) has the logits after 6, the choice after 8, the first gate/up
// products after 21 (7 us of bytes), h at the down units after 24, their products after 27, the last columns combined after 31.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"
#include "route_token.cuh"
#include "tc_gemm.cuh"

namespace invmoe {

namespace {

constexpr int kTok = kDecodeMaxTokens;            // columns of every product
constexpr int kPairs = kDecodeMaxPairs;           // (token, slot) pairs
constexpr int kUnitRows = 128;                    // weight rows of a unit at most
constexpr int kRouterRows = 16;
constexpr int kXBytes = kTok * 128;               // a K block (64 elements) of 16 token rows
constexpr int kStageBytes = 2 * (kUnitRows * 128 + kXBytes);   // weights, then tokens
// K blocks of a stage, by a unit's weight rows: what fills it.
__host__ __device__ constexpr int stage_kb(int rows) { return rows > 64 ? 2 : rows > 32 ? 3 : rows > kRouterRows ? 6 : 8; }
constexpr int kQueue = 4;
constexpr int kTmemCols = 32;                     // two accumulators of 16 columns
constexpr int kStageRow = kUnitRows + 4;          // floats of a staged token column
constexpr int kEpiThreads = 128, kRouteThreads = 32 * kTok;
constexpr int kFirstEpi = 4, kFirstRoute = 8;     // warps: weights, MMA, tokens, -, 4 epilogue, 16 routing
constexpr int kDecodeThreads = 32 * (kFirstRoute + kRouteThreads / 32);
constexpr bool stage_fits(int rows) {
  // its copies, and what a 64- or 128-row MMA reads past its weight rows (accumulator rows that nothing uses)
  return stage_kb(rows) * (rows * 128 + kXBytes) <= kStageBytes &&
         (stage_kb(rows) - 1) * rows * 128 + (rows > 64 ? 128 : 64) * 128 <= kStageBytes;
}
static_assert(stage_fits(128) && stage_fits(96) && stage_fits(64) && stage_fits(32) && stage_fits(kRouterRows), "stage");

enum UnitType : int { kRouter, kSharedUp, kUp, kSharedDown, kDown, kEnd };

// Shared memory: ring, staging, plan, barriers.
template <int EPL>
struct DecodeShape {
  static constexpr int E = EPL * 32;
  static constexpr int STAGING = kTok * kStageRow * 4;
  static constexpr int KEYS = (kRouteThreads / 32) * (E + E / 32 + 1) * 4;
  static constexpr int PLAN = E * (4 + 2) + kPairs * (4 + 2 + 1) + (kPairs + 1) * 2 * 2 + (kRouteThreads / 32) * 4 + 64;
  static constexpr int BARS = 512;
  static constexpr int FIXED = 1024 + STAGING + KEYS + PLAN + BARS;
  static constexpr int STAGES = (232448 - FIXED) / kStageBytes;
  static constexpr int SMEM = FIXED + STAGES * kStageBytes;
  static_assert(STAGES >= 4 && 8 * (2 * STAGES + 2 * kQueue + 8) + 16 * kQueue + 32 + 32 <= BARS, "shared memory");
};

struct Unit {
  int type, expert, slot, tile;                   // slot: index among the chosen experts
};

// One answer for all threads of a named barrier, which orders their shared memory as well.
__device__ __forceinline__ bool bar_and(int id, int threads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "barrier.cta.red.and.pred p, %2, %3, q;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(v ? 1u : 0u), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void bar_named(int id, int threads) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ int load_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void store_release(int* p, int v) {
  asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ int add_acq_rel(int* p, int v) {
  int old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}
// What this thread wrote, and what a barrier ordered before it, is seen by whoever acquires the count.
__device__ __forceinline__ void add_release(int* p, int v) {
  asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// Orders ordinary accesses of global memory and the copies' accesses.
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// Bounded poll until *p >= want; as mbar_wait where it gives up.
__device__ __forceinline__ bool poll_at_least(const int* p, int want, const WaitCtl& w) {
  if (load_acquire(p) >= want) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 0; it < (1u << 28); ++it) {
    if (load_acquire(p) >= want) return true;
    if (*w.abort) return false;
    if (global_timer_ns() - t0 > w.limit_ns) break;
    __nanosleep(20);
  }
  *w.abort = 1;
  atomicOr(w.status, kStatusTimeout);
  return false;
}

// The routing threads' wait: thread 0 tests, all of them go from barrier to barrier.  A multiprocessor whose warps have all
// been waiting for some microseconds comes back slowly: with thread 0 polling and the others at one barrier, the choice of
// one token among 128 experts took 3.3 us after the wait, kept awake like this 1.0 (the layer 33.3 us and 30.1); kept awake
// for the rest of the kernel as well, 28.7, and the GLM-scale layer 109.0 us instead of 110.5.
template <typename F>
__device__ __forceinline__ bool wait_awake(F&& there, int tid, int* s_state, const WaitCtl& w) {
  const uint64_t began = global_timer_ns();
  int state = 0;
  while (state == 0) {
    if (tid == 0) {
      state = there() ? 1 : 0;
      if (state == 0 && (*w.abort || global_timer_ns() - began > w.limit_ns)) {
        if (!*w.abort) atomicOr(w.status, kStatusTimeout);
        *w.abort = 1;
        state = -1;
      }
      *s_state = state;
    }
    bar_named(2, kRouteThreads);
    state = *s_state;
    bar_named(2, kRouteThreads);
  }
  return state > 0;
}

// One lane of a converged warp: what issues copies and MMAs takes its operands from uniform registers.
__device__ __forceinline__ bool elect_lane() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r));
  return r != 0;
}

// 16 consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void reg_fence16(uint32_t (&r)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ void tma_load_w4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

__device__ __forceinline__ void tma_load_w5d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2, int c3,
                                             int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}

template <int I>
using Int = std::integral_constant<int, I>;

// A unit's MMAs: n stages of KB K blocks from `stage` on, K ascending in one accumulation chain.  K blocks past the last (kb)
// are not multiplied.
template <int M, int KB, int STAGES>
__device__ __forceinline__ bool run_unit(uint64_t* full, uint64_t* empty, int stage, uint32_t phase, int n, uint32_t d,
                                         uint64_t desc0, int rows, int kb, const WaitCtl& wc) {
  const uint64_t slice = static_cast<uint64_t>((rows * 128) >> 4);
  for (int st = 0; st < n; ++st) {
    if (!mbar_wait(&full[stage], phase, wc)) return false;
    uint64_t a = desc0 + static_cast<uint64_t>((stage * kStageBytes) >> 4);
    uint64_t b = a + KB * slice;
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      if (st * KB + j < kb) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_bf16(d, a + 2u * kk, b + 2u * kk, idesc_bf16_f32(M, kTok), (st | j | kk) != 0 ? 1u : 0u);
      }
      a += slice;
      b += static_cast<uint64_t>(kXBytes >> 4);
    }
    umma_commit(&empty[stage]);
    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
  }
  return true;
}

// Boxes of stage_kb(rows of the unit) K blocks.
struct DecodeMaps {
  CUtensorMap router, w13, w2, x_router, x, h;     // weight rows (of w13 gate rows and the matching up rows), 16 token rows
  CUtensorMap ws13, ws2, x_shared, hs;             // the shared expert's; not set without one
};

template <int EPL>
__global__ void __launch_bounds__(kDecodeThreads, 1)
    moe_decode_kernel(const __grid_constant__ DecodeMaps maps, const __grid_constant__ DecodeParams p) {
  using S = DecodeShape<EPL>;
  constexpr int STAGES = S::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* stg = reinterpret_cast<float*>(ring + STAGES * kStageBytes);            // [token column][unit row]
  uint32_t* s_keys = reinterpret_cast<uint32_t*>(stg + kTok * kStageRow);
  uint32_t* s_mask = s_keys + S::KEYS / 4;                                       // [E] tokens that chose the expert
  uint32_t* s_scan = s_mask + S::E;                                              // [routing warps]
  float* s_w = reinterpret_cast<float*>(s_scan + kRouteThreads / 32);            // [T * k]
  uint16_t* s_row0 = reinterpret_cast<uint16_t*>(s_w + kPairs);                  // [E] first row in plan order
  uint16_t* s_slot = s_row0 + S::E;                                              // [T * k] row in plan order
  uint16_t* s_expert = s_slot + kPairs;                                          // [chosen + 1] experts, ascending
  uint16_t* s_off = s_expert + kPairs + 1;                                       // [chosen + 1] first row of each
  uint8_t* s_token = reinterpret_cast<uint8_t*>(s_off + kPairs + 1);             // [T * k] token of a row
  uint64_t* bars = reinterpret_cast<uint64_t*>((reinterpret_cast<uintptr_t>(s_token + kPairs) + 15) & ~uintptr_t(15));
  uint64_t* full = bars;                                         // weights and tokens of a stage
  uint64_t* empty = full + STAGES;
  uint64_t* q_full = empty + STAGES;
  uint64_t* q_empty = q_full + kQueue;
  uint64_t* acc_full = q_empty + kQueue;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* plan_bar = acc_empty + 2;
  uint64_t* comb_full = plan_bar + 1;
  uint64_t* comb_empty = comb_full + 1;
  uint64_t* final_bar = comb_empty + 1;
  Unit* s_queue = reinterpret_cast<Unit*>((reinterpret_cast<uintptr_t>(final_bar + 1) + 15) & ~uintptr_t(15));
  uint32_t* misc = reinterpret_cast<uint32_t*>(s_queue + kQueue);
  uint32_t* tmem_slot = misc;
  volatile int* s_abort = reinterpret_cast<volatile int*>(misc + 1);
  int* s_chosen = reinterpret_cast<int*>(misc + 2);
  volatile int* s_tile = reinterpret_cast<volatile int*>(misc + 3);          // columns to combine, -1: none any more
  int* s_ok = reinterpret_cast<int*>(misc + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 2);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kQueue; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 2 + kEpiThreads / 32);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], kEpiThreads / 32);
    }
    mbar_init(plan_bar, 1);
    mbar_init(comb_full, 1);
    mbar_init(comb_empty, kRouteThreads / 32);
    mbar_init(final_bar, 1);
    *s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem_base = *tmem_slot;
  const WaitCtl wc{s_abort, p.status, p.timeout_ns};
  const int n_router = (p.E + kRouterRows - 1) / kRouterRows;
  const int up = p.F / p.up_rows, shared_up = p.Fs / p.shared_rows, hb = (p.H + p.down_rows - 1) / p.down_rows;
  const int shared_down = p.Fs > 0 ? hb : 0;
  int* router_done = p.flags;
  int* y_done = p.flags + 1;                                    // [hb] down units of the chosen experts
  int* ys_done = y_done + hb;                                   // [hb] the shared expert's
  int* hs_done = ys_done + hb;                                  // the shared expert's up units
  int* h_done = hs_done + 1;                                    // [chosen] up units

  // weight rows of a unit
  auto rows_of = [&](int type) {
    return type == kRouter ? kRouterRows : type == kUp ? 2 * p.up_rows : type == kSharedUp ? 2 * p.shared_rows : p.down_rows;
  };
  // K blocks of a unit, in stages
  auto stages_of = [&](int type) {
    const int kb = (type == kDown ? p.F : type == kSharedDown ? p.Fs : p.H) / 64;
    const int per = stage_kb(rows_of(type));
    return (kb + per - 1) / per;
  };

  if (warp == 0) {
    if (elect_lane()) {
      // ---------------------------------------------------------- units and weights
      int stage = 0, fills = 0, q = 0;
      uint32_t phase = 0, q_phase = 0;
      bool planned = false, ok = true;
      int n_up = 0, n_total = 0;
      const int n_free = n_router + shared_up + shared_down;    // units that need no choice
      int u = blockIdx.x;
      while (true) {
        Unit U{kEnd, 0, 0, 0};
        if (u < n_router) {
          U = {kRouter, 0, 0, u};
        } else if (u < n_router + shared_up) {
          U = {kSharedUp, 0, 0, u - n_router};
        } else if (u < n_free) {
          U = {kSharedDown, 0, 0, u - n_router - shared_up};
        } else {
          if (!planned) {
            ok = mbar_wait(plan_bar, 0, wc);
            planned = true;
            n_up = *s_chosen * up;
            n_total = n_up + *s_chosen * hb;
          }
          const int r = u - n_free;
          if (ok && r < n_total) {
            if (r < n_up) U = {kUp, 0, r / up, r % up};
            else U = {kDown, 0, (r - n_up) / hb, (r - n_up) % hb};
            U.expert = s_expert[U.slot];
          }
        }
        if (!ok || !mbar_wait(&q_empty[q], q_phase ^ 1u, wc)) break;
        s_queue[q] = U;
        mbar_arrive(&q_full[q]);
        if (++q == kQueue) { q = 0; q_phase ^= 1u; }
        if (U.type == kEnd) break;
        const int n = stages_of(U.type), rows = rows_of(U.type), per = stage_kb(rows);
        for (int st = 0; st < n; ++st) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, wc)) { ok = false; break; }
          uint8_t* dst = ring + stage * kStageBytes;
          uint64_t* bar = &full[stage];
          // a box counts its full size, rows and blocks past the end (filled with zeros) included
          mbar_arrive_expect_tx(bar, static_cast<uint32_t>(per * 128 * rows));
          if (U.type == kRouter) tma_load_3d(dst, &maps.router, bar, 0, U.tile * kRouterRows, st * per);
          else if (U.type == kUp) tma_load_w5d(dst, &maps.w13, bar, 0, U.tile * p.up_rows, 0, st * per, U.expert);
          else if (U.type == kSharedUp) tma_load_w5d(dst, &maps.ws13, bar, 0, U.tile * p.shared_rows, 0, st * per, 0);
          else if (U.type == kDown) tma_load_w4d(dst, &maps.w2, bar, 0, U.tile * p.down_rows, st * per, U.expert);
          else tma_load_w4d(dst, &maps.ws2, bar, 0, U.tile * p.down_rows, st * per, 0);
          ++fills;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        u = static_cast<int>(gridDim.x) + atomicAdd(p.ctl, 1);
        if (u < 0) u = 0x7fffffff;                              // a workspace that was not zero: no unit, not one before the first
      }
      if (!ok) *s_abort = 1;
      // every copy this thread issued lands before the block can exit (where the other half of a stage never came, the
      // limit is what lets them land)
      const WaitCtl drain{nullptr, p.status, p.timeout_ns};
      for (int s = 0; s < STAGES && s < fills; ++s)
        mbar_wait(&full[s], static_cast<uint32_t>((fills - 1 - s) / STAGES) & 1u, drain);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks the units, so that the compiler knows what is the same in all lanes (a shuffle from lane 0 says
    // so) and keeps descriptors in uniform registers: with one lane reading the queue an MMA took 46 cycles to issue.
    const uint64_t desc0 = sdesc_k_sw128(smem_u32(ring));
    int stage = 0, q = 0, acc = 0;
    uint32_t phase = 0, q_phase = 0, acc_phase = 0;
    bool ok = true;
    while (true) {
      ok = __all_sync(kFull, lane != 0 || mbar_wait(&q_full[q], q_phase, wc));
      if (!ok) break;
      const int type = __shfl_sync(kFull, s_queue[q].type, 0);
      if (lane == 0) mbar_arrive(&q_empty[q]);
      if (++q == kQueue) { q = 0; q_phase ^= 1u; }
      if (type == kEnd) break;
      const int kb = (type == kDown ? p.F : type == kSharedDown ? p.Fs : p.H) / 64;
      const int n = stages_of(type), rows = rows_of(type);
      const uint32_t d = tmem_base + static_cast<uint32_t>(acc * kTok);
      if (elect_lane()) {
        ok = mbar_wait(&acc_empty[acc], acc_phase ^ 1u, wc);
        tc_fence_after();                                        // the epilogue has read this accumulator
        auto run = [&](auto m, auto per) {
          ok = ok && run_unit<m.value, per.value, STAGES>(full, empty, stage, phase, n, d, desc0, rows, kb, wc);
        };
        if (rows > 64) run(Int<128>{}, Int<stage_kb(128)>{});
        else if (rows > 32) run(Int<64>{}, Int<stage_kb(64)>{});
        else if (rows > kRouterRows) run(Int<64>{}, Int<stage_kb(32)>{});
        else run(Int<64>{}, Int<stage_kb(kRouterRows)>{});
        if (ok) umma_commit(&acc_full[acc]);
      }
      if (!__all_sync(kFull, ok)) break;
      phase ^= static_cast<uint32_t>((stage + n) / STAGES) & 1u;
      stage = (stage + n) % STAGES;
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
    if (elect_lane()) {
      if (!ok) *s_abort = 1;
      // every MMA issued here has finished before the block releases TMEM
      umma_commit(final_bar);
      const WaitCtl drain{nullptr, p.status, p.timeout_ns};
      mbar_wait(final_bar, 0, drain);
    }
  } else if (warp == 2) {
    if (elect_lane()) {
      // ---------------------------------------------------------- the tokens' side
      int stage = 0, fills = 0, q = 0;
      uint32_t phase = 0, q_phase = 0;
      bool ok = true;
      while (true) {
        if (!mbar_wait(&q_full[q], q_phase, wc)) { ok = false; break; }
        const Unit U = s_queue[q];
        mbar_arrive(&q_empty[q]);
        if (++q == kQueue) { q = 0; q_phase ^= 1u; }
        if (U.type == kEnd) break;
        int row = 0;
        if (U.type == kDown || U.type == kSharedDown) {
          const bool shared = U.type == kSharedDown;
          // (the shared expert's units do not wait for the choice, which comes after `go`)
          if (shared && !poll_at_least(p.ctl + 2, 1, wc)) { ok = false; break; }
          if (!poll_at_least(shared ? hs_done : h_done + U.slot, shared ? shared_up : up, wc)) { ok = false; break; }
          fence_proxy_async_global();
          if (!shared) row = s_off[U.slot];
        }
        const CUtensorMap* map = U.type == kRouter      ? &maps.x_router
                                 : U.type == kUp        ? &maps.x
                                 : U.type == kSharedUp  ? &maps.x_shared
                                 : U.type == kDown      ? &maps.h
                                                        : &maps.hs;
        const int n = stages_of(U.type), rows = rows_of(U.type), per = stage_kb(rows);
        for (int st = 0; st < n; ++st) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, wc)) { ok = false; break; }
          uint8_t* dst = ring + stage * kStageBytes;
          uint64_t* bar = &full[stage];
          mbar_arrive_expect_tx(bar, static_cast<uint32_t>(per * kXBytes));
          tma_load_3d(dst + per * rows * 128, map, bar, 0, row, st * per);
          ++fills;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
      }
      if (!ok) *s_abort = 1;
      const WaitCtl drain{nullptr, p.status, p.timeout_ns};
      for (int s = 0; s < STAGES && s < fills; ++s)
        mbar_wait(&full[s], static_cast<uint32_t>((fills - 1 - s) / STAGES) & 1u, drain);
    }
  } else if (warp == 3) {
    if (lane < (p.Fs > 0 ? 10 : 6)) tma_prefetch_desc(&maps.router + lane);
    if (blockIdx.x == 0) {
      // the counters of this call; no block looks at any of them before `go`
      const int n = 2 + 2 * hb + min(p.T * p.k, p.E);
      for (int i = lane; i < n; i += 32) p.flags[i] = 0;
      __syncwarp();
      __threadfence();
      if (lane == 0) store_release(p.ctl + 2, 1);
    }
  } else if (warp >= kFirstEpi && warp < kFirstRoute) {
    // ------------------------------------------------------------ epilogue
    // The four warps agree on every unit's fate, so their barriers always meet.
    const int tid = threadIdx.x - kFirstEpi * 32;
    const int w4 = warp - kFirstEpi;                             // TMEM lane quadrant
    int q = 0, acc = 0;
    uint32_t q_phase = 0, acc_phase = 0;
    bool gone = false;                                           // `go` seen
    uint32_t c_phase = 0;
    auto request = [&](int tile) {                               // thread 0
      if (!mbar_wait(comb_empty, c_phase ^ 1u, wc)) return;
      *s_tile = tile;
      mbar_arrive(comb_full);
      c_phase ^= 1u;
    };
    while (true) {
      // one thread waits, the others at the barrier
      bool ok = true;
      if (tid == 0) {
        ok = mbar_wait(&q_full[q], q_phase, wc);
        if (ok && s_queue[q].type != kEnd) ok = mbar_wait(&acc_full[acc], acc_phase, wc);
        if (ok && !gone) ok = gone = poll_at_least(p.ctl + 2, 1, wc);   // before this block's first count
      }
      if (!bar_and(1, kEpiThreads, ok)) break;
      const Unit U = s_queue[q];
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_empty[q]);
      if (++q == kQueue) { q = 0; q_phase ^= 1u; }
      if (U.type == kEnd) {
        if (tid == 0) request(-1);
        break;
      }
      tc_fence_after();
      uint32_t r[16];
      tmem_ld16(tmem_base + (static_cast<uint32_t>(w4 * 32) << 16) + static_cast<uint32_t>(acc * kTok), r);
      tmem_ld_wait();
      reg_fence16(r);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[acc]);
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      if (U.type == kRouter) {
        // accumulator row 16q + L in lane L < 16 of quadrant q: the 16 experts are quadrant 0's
        const int e = U.tile * kRouterRows + lane;
        if (w4 == 0) {
          if (lane < kRouterRows && e < p.E) {
#pragma unroll
            for (int t = 0; t < kTok; ++t)
              if (t < p.T) p.logits[t * p.E + e] = __uint_as_float(r[t]);
          }
          __syncwarp();
          if (lane == 0) add_release(router_done, 1);
        }
        continue;
      }
      // accumulator rows: one per lane, or (at most 64 rows) 16q + L in lane L < 16 of quadrant q
      const bool wide = rows_of(U.type) > 64;
      if (wide || lane < 16) {
        const int row = wide ? w4 * 32 + lane : w4 * 16 + lane;
#pragma unroll
        for (int t = 0; t < kTok; ++t) stg[t * kStageRow + row] = __uint_as_float(r[t]);
      }
      bar_named(1, kEpiThreads);
      const bool shared = U.type == kSharedUp || U.type == kSharedDown;
      const int off = shared ? 0 : s_off[U.slot];   // (a unit of a chosen expert comes after the plan)
      const int count = shared ? p.T : s_off[U.slot + 1] - off;
      if (U.type == kUp || U.type == kSharedUp) {
        __nv_bfloat16* out = shared ? p.hs : p.h;
        const int ld = shared ? p.Fs : p.F, rows = shared ? p.shared_rows : p.up_rows;
        if (2 * lane < rows)
          for (int j = w4; j < count; j += 4) {
            const int t = shared ? j : s_token[off + j];
            const float2 g = *reinterpret_cast<const float2*>(stg + t * kStageRow + 2 * lane);
            const float2 v = *reinterpret_cast<const float2*>(stg + t * kStageRow + rows + 2 * lane);
            *reinterpret_cast<uint32_t*>(out + static_cast<long long>(off + j) * ld + U.tile * rows + 2 * lane) =
                pack_bf16x2(__fmul_rn(silu_f32(g.x), v.x), __fmul_rn(silu_f32(g.y), v.y));
          }
        fence_proxy_async_global();                              // read by other blocks' copies
        bar_named(1, kEpiThreads);
        if (tid == 0) add_release(shared ? hs_done : h_done + U.slot, 1);
      } else {
        float* out = shared ? p.ys : p.y;
        const int c = U.tile * p.down_rows + 4 * lane;
        if (4 * lane < p.down_rows && c < p.H)
          for (int j = w4; j < count; j += 4)
            *reinterpret_cast<float4*>(out + static_cast<long long>(off + j) * p.H + c) =
                *reinterpret_cast<const float4*>(stg + j * kStageRow + 4 * lane);
        bar_named(1, kEpiThreads);
        // the last of the chosen experts' blocks of these columns: the routing warps combine them
        if (tid == 0) {
          if (shared) add_release(ys_done + U.tile, 1);
          else if (add_acq_rel(y_done + U.tile, 1) == *s_chosen - 1) request(U.tile);
        }
      }
    }
  } else if (warp >= kFirstRoute) {
    // ------------------------------------------------------------ the choice, by every block for itself: a warp per token
    const int tid = threadIdx.x - kFirstRoute * 32;
    const int t = warp - kFirstRoute;
    static_assert(S::E <= kRouteThreads, "a thread per expert");
    if (tid < S::E) s_mask[tid] = 0u;
    if (wait_awake([&] { return load_acquire(p.ctl + 2) >= 1 && load_acquire(router_done) >= n_router; }, tid, s_ok, wc)) {
      const float* row = p.logits + t * p.E;
      const LoadL2 ld{};
      const SelectParams sp{row, p.bias, p.T, p.E, p.k, p.n_group, p.topk_group, p.renorm, p.scale, nullptr, nullptr};
      SoftmaxStats stats;
      int e = 0;
      float v = 0.0f;
      if (t < p.T) {
        const bool groups = p.n_group > 1;
        uint32_t* keys = s_keys + t * (S::E + S::E / 32 + 1);
        if (p.score == kDecodeTopk)
          topk_choose<EPL>(row, ld, p.E, p.k, lane, e, v);
        else if (p.score == kDecodeSigmoid)
          groups ? select_choose<EPL, false, true>(row, ld, sp, keys, lane, e, stats)
                 : select_choose<EPL, false, false>(row, ld, sp, keys, lane, e, stats);
        else
          groups ? select_choose<EPL, true, true>(row, ld, sp, keys, lane, e, stats)
                 : select_choose<EPL, true, false>(row, ld, sp, keys, lane, e, stats);
        if (lane < p.k) atomicOr(&s_mask[e], 1u << t);
      }
      bar_named(2, kRouteThreads);
      // a thread per expert: chosen ones ascending, each with its rows, tokens ascending; rows and experts in one sum
      const uint32_t mask = tid < S::E ? s_mask[tid] : 0u;
      const uint32_t mine = static_cast<uint32_t>(__popc(mask)) << 16 | (mask != 0u ? 1u : 0u);
      uint32_t sum = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(kFull, sum, d);
        if (lane >= d) sum += o;
      }
      if (lane == 31) s_scan[t] = sum;
      bar_named(2, kRouteThreads);
      uint32_t all = 0u;
      for (int w = 0; w < kRouteThreads / 32; ++w) {
        if (w == t) sum += all;
        all += s_scan[w];
      }
      if (mask != 0u) {
        int r = static_cast<int>((sum - mine) >> 16);
        const int a = static_cast<int>((sum - mine) & 0xffffu);
        s_expert[a] = static_cast<uint16_t>(tid);
        s_off[a] = static_cast<uint16_t>(r);
        s_row0[tid] = static_cast<uint16_t>(r);
        for (uint32_t m = mask; m != 0u; m &= m - 1u) s_token[r++] = static_cast<uint8_t>(__ffs(m) - 1);
      }
      if (tid == 0) {
        *s_chosen = static_cast<int>(all & 0xffffu);
        s_off[all & 0xffffu] = static_cast<uint16_t>(all >> 16);
      }
      bar_named(2, kRouteThreads);
      if (tid == 0) mbar_arrive(plan_bar);
      // the units are on their way; weights and rows of the pairs are for the combine
      if (t < p.T) {
        const float w = p.score == kDecodeTopk      ? topk_gate(v, p.k, lane)
                        : p.score == kDecodeSigmoid ? select_weight<false>(row, ld, sp, e, stats, lane)
                                                    : select_weight<true>(row, ld, sp, e, stats, lane);
        if (lane < p.k) {
          const int i = t * p.k + lane;
          s_w[i] = w;
          s_slot[i] = static_cast<uint16_t>(s_row0[e] + __popc(s_mask[e] & ((1u << t) - 1u)));
          if (blockIdx.x == 0) {
            if (p.topk_idx != nullptr) p.topk_idx[i] = e;
            if (p.topk_w != nullptr) p.topk_w[i] = w;
          }
        }
      }
      __syncwarp();
      // columns whose last unit this block finished: out = ((w0 y0 + w1 y1) + ...) + y_shared, every product and sum
      // rounded; the warp's token, with the loads of eight slots in flight
      uint32_t c_phase = 0;
      while (wait_awake([&] { return mbar_test(comb_full, c_phase); }, tid, s_ok, wc)) {
        const int tile = *s_tile;
        __syncwarp();
        if (lane == 0) mbar_arrive(comb_empty);
        c_phase ^= 1u;
        if (tile < 0) break;
        const int c = tile * p.down_rows + 4 * lane;
        if (t >= p.T) continue;
        if (p.Fs > 0) {
          if (!__all_sync(kFull, lane != 0 || poll_at_least(ys_done + tile, 1, wc))) continue;   // (the next wait fails too)
          __syncwarp();
        }
        if (4 * lane >= p.down_rows || c >= p.H) continue;
        const long long at = static_cast<long long>(t) * p.H + c;
        float4 a, sh = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.Fs > 0) sh = __ldcg(reinterpret_cast<const float4*>(p.ys + at));
        for (int j0 = 0; j0 < p.k; j0 += 8) {
          float4 y[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j0 + j < p.k)
              y[j] = __ldcg(reinterpret_cast<const float4*>(p.y + static_cast<long long>(s_slot[t * p.k + j0 + j]) * p.H + c));
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (j0 + j < p.k) {
              const float wj = s_w[t * p.k + j0 + j];
              const float4 m = make_float4(__fmul_rn(wj, y[j].x), __fmul_rn(wj, y[j].y), __fmul_rn(wj, y[j].z),
                                           __fmul_rn(wj, y[j].w));
              a = (j0 | j) == 0 ? m : make_float4(__fadd_rn(a.x, m.x), __fadd_rn(a.y, m.y), __fadd_rn(a.z, m.z),
                                                  __fadd_rn(a.w, m.w));
            }
          }
        }
        if (p.Fs > 0) a = make_float4(__fadd_rn(a.x, sh.x), __fadd_rn(a.y, sh.y), __fadd_rn(a.z, sh.z), __fadd_rn(a.w, sh.w));
        if (p.out != nullptr) *reinterpret_cast<float4*>(p.out + at) = a;
        if (p.out_bf16 != nullptr)
          *reinterpret_cast<uint2*>(p.out_bf16 + at) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
      }
    }
  }

  __syncwarp();                                                  // the elected lanes rejoin their warps
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
  if (threadIdx.x == 0) {
    // the last block leaves the words of the status block as it found them
    __threadfence();
    if (atomicAdd(p.ctl + 1, 1) == static_cast<int>(gridDim.x) - 1) {
      p.ctl[0] = 0;
      p.ctl[1] = 0;
      p.ctl[2] = 0;
      __threadfence();
    }
  }
}

// [E][2F][K] bf16 (gate rows, then up rows) as (64, F rows, gate/up, K / 64, E): a box holds `rows` gate rows and the
// matching up rows.
int make_tmap_up(CUtensorMap* m, const void* base, long long K, long long F, long long E, unsigned rows) {
  const unsigned long long dims[5] = {64, static_cast<unsigned long long>(F), 2, static_cast<unsigned long long>(K / 64),
                                      static_cast<unsigned long long>(E)};
  const unsigned long long strides[4] = {2ull * K, 2ull * K * F, 128, 4ull * K * F};
  const unsigned box[5] = {64, rows, 2, static_cast<unsigned>(stage_kb(2 * rows)), 1};
  return make_tmap_bf16(m, base, 5, dims, strides, box);
}

// [E][N][K] bf16 as (64, N rows, K / 64, E): a box holds `rows` rows.
int make_tmap_down(CUtensorMap* m, const void* base, long long K, long long N, long long E, unsigned rows) {
  const unsigned long long dims[4] = {64, static_cast<unsigned long long>(N), static_cast<unsigned long long>(K / 64),
                                      static_cast<unsigned long long>(E)};
  const unsigned long long strides[3] = {2ull * K, 128, 2ull * K * N};
  const unsigned box[4] = {64, rows, static_cast<unsigned>(stage_kb(rows)), 1};
  return make_tmap_bf16(m, base, 4, dims, strides, box);
}

// [rows][K] bf16 as (64, rows, K / 64): box_rows rows of `blocks` K blocks.
int make_tmap_rows(CUtensorMap* m, const void* base, long long K, long long rows, unsigned box_rows, int blocks) {
  const unsigned long long dims[3] = {64, static_cast<unsigned long long>(rows), static_cast<unsigned long long>(K / 64)};
  const unsigned long long strides[2] = {2ull * K, 128};
  const unsigned box[3] = {64, box_rows, static_cast<unsigned>(blocks)};
  return make_tmap_bf16(m, base, 3, dims, strides, box);
}

// Rows of a unit, for `experts` times `total` rows: the largest size, or where that gives a block two units at most the one
// with the fewest rows for the busiest block.
int unit_rows(long long experts, int total, int sms, std::initializer_list<int> sizes) {
  int best = 0;
  long long best_cost = 0;
  for (int r : sizes) {
    if (total % r != 0 && total > r) continue;
    const long long units = experts * ((total + r - 1) / r);
    const long long cost = (units + sms - 1) / sms * r;
    if (best != 0 && best_cost > 2 * best) break;
    if (best == 0 || cost < best_cost) {
      best = r;
      best_cost = cost;
    }
  }
  return best;
}

template <int EPL>
int launch_decode(const DecodeCall& c, DecodeParams p, cudaStream_t st) {
  using S = DecodeShape<EPL>;
  int sms = 0;
  int rc = device_sm_count(&sms);
  if (rc) return rc;
  const long long experts = p.T * p.k < p.E ? p.T * p.k : p.E;
  p.up_rows = unit_rows(experts, p.F, sms, {64, 48, 32});
  p.shared_rows = p.Fs > 0 ? unit_rows(1, p.Fs, sms, {64, 32, 16}) : 64;
  p.down_rows = unit_rows(experts, p.H, sms, {128, 64});
  const unsigned ur = p.up_rows, sr = p.shared_rows, dr = p.down_rows;
  DecodeMaps m{};
  rc = make_tmap_rows(&m.router, c.w_router, p.H, p.E, kRouterRows, stage_kb(kRouterRows));
  if (!rc) rc = make_tmap_rows(&m.x_router, c.x, p.H, p.T, kTok, stage_kb(kRouterRows));
  if (!rc) rc = make_tmap_rows(&m.x, c.x, p.H, p.T, kTok, stage_kb(2 * p.up_rows));
  if (!rc) rc = make_tmap_rows(&m.h, p.h, p.F, p.T * p.k, kTok, stage_kb(p.down_rows));
  if (!rc) rc = make_tmap_up(&m.w13, c.w13, p.H, p.F, p.E, ur);
  if (!rc) rc = make_tmap_down(&m.w2, c.w2, p.F, p.H, p.E, dr);
  if (!rc && p.Fs > 0) {
    rc = make_tmap_rows(&m.x_shared, c.x, p.H, p.T, kTok, stage_kb(2 * p.shared_rows));
    if (!rc) rc = make_tmap_rows(&m.hs, p.hs, p.Fs, p.T, kTok, stage_kb(p.down_rows));
    if (!rc) rc = make_tmap_up(&m.ws13, c.ws13, p.H, p.Fs, 1, sr);
    if (!rc) rc = make_tmap_down(&m.ws2, c.ws2, p.Fs, p.H, 1, dr);
  }
  static std::atomic<uint64_t> attr_set{0};
  if (!rc) rc = set_smem_attr(reinterpret_cast<const void*>(moe_decode_kernel<EPL>), S::SMEM, attr_set);
  if (rc) return rc;
  // as many blocks as the largest phase has units, one to an SM
  const long long hb = (p.H + p.down_rows - 1) / p.down_rows;
  long long units = experts * (p.F / p.up_rows);
  if (experts * hb > units) units = experts * hb;
  const long long first = (p.E + kRouterRows - 1) / kRouterRows + (p.Fs > 0 ? p.Fs / p.shared_rows + hb : 0);
  if (first > units) units = first;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units < sms ? units : sms));
  cfg.blockDim = dim3(kDecodeThreads);
  cfg.dynamicSmemBytes = S::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;                   // blocks wait for one another: all are resident
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  ProfScope prof("moe_decode", st);
  return check_cuda(cudaLaunchKernelEx(&cfg, moe_decode_kernel<EPL>, m, p), "moe_decode_kernel");
}

}  // namespace

int moe_decode_launch(const DecodeCall& c, const DecodeParams& p, cudaStream_t st) {
  return p.E <= 128 ? launch_decode<4>(c, p, st) : p.E <= 256 ? launch_decode<8>(c, p, st) : launch_decode<16>(c, p, st);
}

}  // namespace invmoe
