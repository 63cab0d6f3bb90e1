// moe_decode.cu -- the whole MoE layer of at most 16 tokens in one kernel (sm_103a).
//
//   l = x Wr^T;  experts and weights of each token from l;  h_e = bf16(silu(x Wg_e) (x Wu_e));  y_e = h_e Wd_e;
//   out = sum_j weight_j y_j + y_shared
//
// Bound by reading the weights of the experts that some token chose, once.  As a chain of kernels (moe_layer_forward) every
// product ends in a partly filled wave and every launch in a gap; here one persistent, cooperatively launched kernel walks
// one list of units, largest first, taken from a counter:
//     router (16 experts), shared gate/up, | gate/up of the chosen experts, shared down, down of the chosen experts
// A unit is 64 gate rows with the matching 64 up rows, or 128 rows of the down projection, over their whole K; what is
// behind the bar needs the choice.  Weights stream through a shared-memory ring ahead of every dependency: one thread loads
// weights as soon as a stage is free, another one the tokens' side, and only that one waits until h is there.  Waits are
// bounded polls of counters in the workspace: the router's units done (then every block makes the choice for itself, from
// the logits, into shared memory), an expert's gate/up units done.  No block waits for a unit that the counter has not handed
// out before its own, and a cooperative launch keeps all blocks resident, so every wait ends.  The block that finishes a
// column of 128 outputs combines it, in rank order.
//
// The tensor cores do the products although a unit of 16 tokens keeps them nearly idle: an element's bits are those of the
// other engines (K ascending in K = 16 steps of one accumulation chain, no split), so a token's output here is, bit for bit,
// what moe_layer_forward gives it in any batch.  Weights are the MMA's M side (128 rows; 64, of which 16 are used, for the
// router, whose chain of K / 16 dependent MMAs is what everything else waits for), the tokens its N side, all 16 columns of
// it: gate/up takes x as it is and keeps the columns of the tokens that chose the expert.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"
#include "route_token.cuh"
#include "tc_gemm.cuh"

namespace invmoe {

namespace {

constexpr int kTok = kDecodeMaxTokens;            // columns of every product
constexpr int kPairs = kDecodeMaxPairs;           // (token, slot) pairs
constexpr int kUnitRows = 128;
constexpr int kRouterRows = 16;
constexpr int kRouterKb = 4;                      // K blocks of a router stage
constexpr int kWBytes = kUnitRows * 128;          // a K block (64 elements) of a unit's weights
constexpr int kXBytes = kTok * 128;               // a K block of 16 token rows
constexpr int kStageBytes = kWBytes + kXBytes;
constexpr int kQueue = 4;
constexpr int kTmemCols = 32;                     // two accumulators of 16 columns
constexpr int kStageRow = kUnitRows + 4;          // floats of a staged token column
constexpr int kEpiThreads = 128, kRouteThreads = 256;
constexpr int kFirstEpi = 4, kFirstRoute = 8;     // warps: weights, MMA, tokens, -, 4 epilogue, 8 routing
constexpr int kDecodeThreads = 32 * (kFirstRoute + kRouteThreads / 32);
static_assert(kRouterKb * (kRouterRows * 128 + kXBytes) <= kStageBytes, "router stage");
static_assert((kRouterKb - 1) * kRouterRows * 128 + 64 * 128 <= kStageBytes, "what the 64-row MMA reads past its 16 rows");

enum UnitType : int { kRouter, kSharedUp, kUp, kSharedDown, kDown, kEnd };

// Shared memory: ring, staging, plan, barriers.
template <int EPL>
struct DecodeShape {
  static constexpr int E = EPL * 32;
  static constexpr int STAGING = kTok * kStageRow * 4;
  static constexpr int KEYS = (kRouteThreads / 32) * (E + E / 32 + 1) * 4;
  static constexpr int PLAN = E * 4 + kPairs * (2 + 4 + 2 + 1) + (kPairs + 1) * 2 * 2 + 64;
  static constexpr int BARS = 512;
  static constexpr int FIXED = 1024 + STAGING + KEYS + PLAN + BARS;
  static constexpr int STAGES = (232448 - FIXED) / kStageBytes;
  static constexpr int SMEM = FIXED + STAGES * kStageBytes;
  static_assert(STAGES >= 6 && 8 * (3 * STAGES + 2 * kQueue + 6) + 16 * kQueue + 32 <= BARS, "shared memory");
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
// Order writes of this thread's (or, after a barrier, its block's) generic proxy and the async proxy's reads of global memory.
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

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

struct DecodeMaps {
  CUtensorMap router, x_router;   // boxes of kRouterKb K blocks
  CUtensorMap x, h, hs;           // 16 rows, one K block
  CUtensorMap w13, ws13;          // 64 gate and 64 up rows, one K block
  CUtensorMap w2, ws2;            // 128 rows, one K block
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
  float* s_w = reinterpret_cast<float*>(s_mask + S::E);                          // [T * k]
  uint16_t* s_idx = reinterpret_cast<uint16_t*>(s_w + kPairs);                   // [T * k] expert
  uint16_t* s_slot = s_idx + kPairs;                                             // [T * k] row in plan order
  uint16_t* s_expert = s_slot + kPairs;                                          // [chosen + 1] experts, ascending
  uint16_t* s_off = s_expert + kPairs + 1;                                       // [chosen + 1] first row of each
  uint8_t* s_token = reinterpret_cast<uint8_t*>(s_off + kPairs + 1);             // [T * k] token of a row
  uint64_t* bars = reinterpret_cast<uint64_t*>((reinterpret_cast<uintptr_t>(s_token + kPairs) + 15) & ~uintptr_t(15));
  uint64_t* full_w = bars;
  uint64_t* full_x = full_w + STAGES;
  uint64_t* empty = full_x + STAGES;
  uint64_t* q_full = empty + STAGES;
  uint64_t* q_empty = q_full + kQueue;
  uint64_t* acc_full = q_empty + kQueue;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* plan_bar = acc_empty + 2;
  uint64_t* final_bar = plan_bar + 1;
  Unit* s_queue = reinterpret_cast<Unit*>((reinterpret_cast<uintptr_t>(final_bar + 1) + 15) & ~uintptr_t(15));
  uint32_t* misc = reinterpret_cast<uint32_t*>(s_queue + kQueue);
  uint32_t* tmem_slot = misc;
  volatile int* s_abort = reinterpret_cast<volatile int*>(misc + 1);
  int* s_chosen = reinterpret_cast<int*>(misc + 2);
  int* s_last = reinterpret_cast<int*>(misc + 3);
  int* s_ok = reinterpret_cast<int*>(misc + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full_w[s], 1);
      mbar_init(&full_x[s], 1);
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
    mbar_init(final_bar, 1);
    *s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
  if (blockIdx.x == 0 && warp == 3) {
    // the counters of this call; the other blocks look at none of them before `go`
    for (int i = lane; i < kDecodeFlags; i += 32) p.flags[i] = 0;
    __syncwarp();
    __threadfence();
    if (lane == 0) store_release(p.ctl + 2, 1);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem_base = *tmem_slot;
  const WaitCtl wc{s_abort, p.status, p.timeout_ns};
  int* router_done = p.flags;
  int* y_done = p.flags + 1;                                    // [hb]
  int* h_done = y_done + kDecodeMaxBlocks;                      // [chosen], the shared expert's last
  const int n_router = (p.E + kRouterRows - 1) / kRouterRows;
  const int up = p.F / 64, shared_up = p.Fs / 64, hb = (p.H + kUnitRows - 1) / kUnitRows;

  // K blocks of a unit, in stages
  auto stages_of = [&](int type) {
    const int kb = (type == kDown ? p.F : type == kSharedDown ? p.Fs : p.H) / 64;
    return type == kRouter ? (kb + kRouterKb - 1) / kRouterKb : kb;
  };

  if (warp == 0) {
    if (elect_lane()) {
      // ---------------------------------------------------------- units and weights
      int stage = 0, fills = 0, q = 0;
      uint32_t phase = 0, q_phase = 0;
      bool planned = false, ok = true;
      int n_up = 0, n_total = 0;
      const int n_free = n_router + shared_up;                  // units that need no choice
      int u = blockIdx.x;
      while (true) {
        Unit U{kEnd, 0, 0, 0};
        if (u < n_router) {
          U = {kRouter, 0, 0, u};
        } else if (u < n_free) {
          U = {kSharedUp, 0, 0, u - n_router};
        } else {
          if (!planned) {
            ok = mbar_wait(plan_bar, 0, wc);
            planned = true;
            n_up = *s_chosen * up;
            n_total = n_up + (p.Fs > 0 ? hb : 0) + *s_chosen * hb;
          }
          int r = u - n_free;
          if (ok && r < n_total) {
            if (r < n_up) {
              U = {kUp, 0, r / up, r % up};
            } else if ((r -= n_up) < (p.Fs > 0 ? hb : 0)) {
              U = {kSharedDown, 0, 0, r};
            } else {
              r -= p.Fs > 0 ? hb : 0;
              U = {kDown, 0, r / hb, r % hb};
            }
            if (U.type != kSharedDown) U.expert = s_expert[U.slot];
          }
        }
        if (!ok || !mbar_wait(&q_empty[q], q_phase ^ 1u, wc)) break;
        s_queue[q] = U;
        mbar_arrive(&q_full[q]);
        if (++q == kQueue) { q = 0; q_phase ^= 1u; }
        if (U.type == kEnd) break;
        const int n = stages_of(U.type);
        for (int st = 0; st < n; ++st) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, wc)) { ok = false; break; }
          uint8_t* dst = ring + stage * kStageBytes;
          uint64_t* bar = &full_w[stage];
          if (U.type == kRouter) {
            mbar_arrive_expect_tx(bar, kRouterKb * kRouterRows * 128);
            tma_load_3d(dst, &maps.router, bar, 0, U.tile * kRouterRows, st * kRouterKb);
          } else {
            mbar_arrive_expect_tx(bar, kWBytes);
            if (U.type == kUp) tma_load_w4d(dst, &maps.w13, bar, st * 64, U.tile * 64, 0, U.expert);
            else if (U.type == kSharedUp) tma_load_w4d(dst, &maps.ws13, bar, st * 64, U.tile * 64, 0, 0);
            else if (U.type == kDown) tma_load_3d(dst, &maps.w2, bar, st * 64, U.tile * kUnitRows, U.expert);
            else tma_load_3d(dst, &maps.ws2, bar, st * 64, U.tile * kUnitRows, 0);
          }
          ++fills;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        u = static_cast<int>(gridDim.x) + atomicAdd(p.ctl, 1);
      }
      if (!ok) *s_abort = 1;
      // every copy this thread issued lands before the block can exit
      const WaitCtl drain{nullptr, p.status, p.timeout_ns};
      for (int s = 0; s < STAGES && s < fills; ++s)
        mbar_wait(&full_w[s], static_cast<uint32_t>((fills - 1 - s) / STAGES) & 1u, drain);
    }
  } else if (warp == 1) {
    if (elect_lane()) {
      // ---------------------------------------------------------- MMA issuer
      const uint64_t desc0 = sdesc_k_sw128(smem_u32(ring));
      int stage = 0, q = 0, acc = 0;
      uint32_t phase = 0, q_phase = 0, acc_phase = 0;
      bool ok = true;
      while (true) {
        if (!mbar_wait(&q_full[q], q_phase, wc)) { ok = false; break; }
        const int type = s_queue[q].type;
        mbar_arrive(&q_empty[q]);
        if (++q == kQueue) { q = 0; q_phase ^= 1u; }
        if (type == kEnd) break;
        if (!mbar_wait(&acc_empty[acc], acc_phase ^ 1u, wc)) { ok = false; break; }
        const int n = stages_of(type);
        const int kb_all = p.H / 64;
        const uint32_t d = tmem_base + static_cast<uint32_t>(acc * kTok);
        for (int st = 0; st < n; ++st) {
          if (!mbar_wait(&full_w[stage], phase, wc) || !mbar_wait(&full_x[stage], phase, wc)) { ok = false; break; }
          tc_fence_after();
          const uint64_t a = desc0 + static_cast<uint64_t>((stage * kStageBytes) >> 4);
          if (type == kRouter) {
            const uint64_t b = a + static_cast<uint64_t>((kRouterKb * kRouterRows * 128) >> 4);
            const int blocks = min(kRouterKb, kb_all - st * kRouterKb);
            for (int j = 0; j < blocks; ++j)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_bf16(d, a + static_cast<uint64_t>(j * ((kRouterRows * 128) >> 4)) + 2u * kk,
                          b + static_cast<uint64_t>(j * (kXBytes >> 4)) + 2u * kk, idesc_bf16_f32(64, kTok),
                          (st | j | kk) != 0 ? 1u : 0u);
          } else {
            const uint64_t b = a + static_cast<uint64_t>(kWBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_bf16(d, a + 2u * kk, b + 2u * kk, idesc_bf16_f32(kUnitRows, kTok), (st | kk) != 0 ? 1u : 0u);
          }
          umma_commit(&empty[stage]);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        umma_commit(&acc_full[acc]);
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
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
          if (!poll_at_least(h_done + (shared ? kPairs : U.slot), shared ? shared_up : up, wc)) { ok = false; break; }
          fence_proxy_async_all();
          if (!shared) row = s_off[U.slot];
        }
        const int n = stages_of(U.type);
        for (int st = 0; st < n; ++st) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, wc)) { ok = false; break; }
          uint8_t* dst = ring + stage * kStageBytes;
          uint64_t* bar = &full_x[stage];
          if (U.type == kRouter) {
            mbar_arrive_expect_tx(bar, kRouterKb * kXBytes);
            tma_load_3d(dst + kRouterKb * kRouterRows * 128, &maps.x_router, bar, 0, 0, st * kRouterKb);
          } else {
            mbar_arrive_expect_tx(bar, kXBytes);
            const CUtensorMap* map = U.type == kDown ? &maps.h : U.type == kSharedDown ? &maps.hs : &maps.x;
            tma_load_2d(dst + kWBytes, map, bar, st * 64, row);
          }
          ++fills;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
      }
      if (!ok) *s_abort = 1;
      const WaitCtl drain{nullptr, p.status, p.timeout_ns};
      for (int s = 0; s < STAGES && s < fills; ++s)
        mbar_wait(&full_x[s], static_cast<uint32_t>((fills - 1 - s) / STAGES) & 1u, drain);
    }
  } else if (warp >= kFirstEpi && warp < kFirstRoute) {
    // ------------------------------------------------------------ epilogue
    // The four warps agree on every unit's fate, so their barriers always meet.
    const int tid = threadIdx.x - kFirstEpi * 32;
    const int w4 = warp - kFirstEpi;                             // TMEM lane quadrant
    int q = 0, acc = 0;
    uint32_t q_phase = 0, acc_phase = 0;
    bool gone = false;                                           // `go` seen
    while (true) {
      bool ok = mbar_wait(&q_full[q], q_phase, wc);
      Unit U{kEnd, 0, 0, 0};
      if (ok) U = s_queue[q];
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&q_empty[q]);
      if (++q == kQueue) { q = 0; q_phase ^= 1u; }
      if (ok && U.type != kEnd) ok = mbar_wait(&acc_full[acc], acc_phase, wc);
      if (!gone && ok && tid == 0) {
        ok = poll_at_least(p.ctl + 2, 1, wc);                    // before this block's first count
        gone = ok;
      }
      if (!bar_and(1, kEpiThreads, ok)) break;
      if (U.type == kEnd) break;
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
          __threadfence();
          __syncwarp();
          if (lane == 0) add_acq_rel(router_done, 1);
        }
        continue;
      }
#pragma unroll
      for (int t = 0; t < kTok; ++t) stg[t * kStageRow + w4 * 32 + lane] = __uint_as_float(r[t]);
      bar_named(1, kEpiThreads);
      const bool shared = U.type == kSharedUp || U.type == kSharedDown;
      const int off = shared ? 0 : s_off[U.slot];
      const int count = shared ? p.T : s_off[U.slot + 1] - off;
      if (U.type == kUp || U.type == kSharedUp) {
        __nv_bfloat16* out = shared ? p.hs : p.h;
        const int ld = shared ? p.Fs : p.F;
        for (int j = w4; j < count; j += 4) {
          const int t = shared ? j : s_token[off + j];
          const float2 g = *reinterpret_cast<const float2*>(stg + t * kStageRow + 2 * lane);
          const float2 v = *reinterpret_cast<const float2*>(stg + t * kStageRow + 64 + 2 * lane);
          *reinterpret_cast<uint32_t*>(out + static_cast<long long>(off + j) * ld + U.tile * 64 + 2 * lane) =
              pack_bf16x2(__fmul_rn(silu_f32(g.x), v.x), __fmul_rn(silu_f32(g.y), v.y));
        }
        fence_proxy_async_all();                                 // read by other blocks' copies
        __threadfence();
        bar_named(1, kEpiThreads);
        if (tid == 0) {
          fence_proxy_async_all();
          add_acq_rel(h_done + (shared ? kPairs : U.slot), 1);
        }
      } else {
        float* out = shared ? p.ys : p.y;
        const int c = U.tile * kUnitRows + 4 * lane;
        if (c < p.H)
          for (int j = w4; j < count; j += 4)
            *reinterpret_cast<float4*>(out + static_cast<long long>(off + j) * p.H + c) =
                *reinterpret_cast<const float4*>(stg + j * kStageRow + 4 * lane);
        __threadfence();
        bar_named(1, kEpiThreads);
        if (tid == 0) *s_last = add_acq_rel(y_done + U.tile, 1) == *s_chosen + (p.Fs > 0 ? 1 : 0) - 1;
        bar_named(1, kEpiThreads);
        if (*s_last) {
          // this block was the column's last: out = ((w0 y0 + w1 y1) + ...) + y_shared, every product and sum rounded
          __threadfence();
          if (c < p.H) {
            for (int t = w4; t < p.T; t += 4) {
              float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
              for (int j = 0; j < p.k; ++j) {
                const float wj = s_w[t * p.k + j];
                const float4 v = __ldcg(reinterpret_cast<const float4*>(
                    p.y + static_cast<long long>(s_slot[t * p.k + j]) * p.H + c));
                const float4 m = make_float4(__fmul_rn(wj, v.x), __fmul_rn(wj, v.y), __fmul_rn(wj, v.z), __fmul_rn(wj, v.w));
                a = j == 0 ? m : make_float4(__fadd_rn(a.x, m.x), __fadd_rn(a.y, m.y), __fadd_rn(a.z, m.z), __fadd_rn(a.w, m.w));
              }
              const long long at = static_cast<long long>(t) * p.H + c;
              if (p.Fs > 0) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(p.ys + at));
                a = make_float4(__fadd_rn(a.x, v.x), __fadd_rn(a.y, v.y), __fadd_rn(a.z, v.z), __fadd_rn(a.w, v.w));
              }
              if (p.out != nullptr) *reinterpret_cast<float4*>(p.out + at) = a;
              if (p.out_bf16 != nullptr)
                *reinterpret_cast<uint2*>(p.out_bf16 + at) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
            }
          }
        }
      }
    }
  } else if (warp >= kFirstRoute) {
    // ------------------------------------------------------------ the choice, by every block for itself
    const int tid = threadIdx.x - kFirstRoute * 32;
    const int wr = warp - kFirstRoute;
    const int pairs = p.T * p.k;
    for (int e = tid; e < S::E; e += kRouteThreads) s_mask[e] = 0u;
    if (tid == 0) *s_ok = poll_at_least(p.ctl + 2, 1, wc) && poll_at_least(router_done, n_router, wc);
    bar_named(2, kRouteThreads);
    if (*s_ok) {
      for (int t = wr; t < p.T; t += kRouteThreads / 32) {
        const float* row = p.logits + static_cast<long long>(t) * p.E;
        int e = 0;
        float w = 0.0f;
        if (p.score == kDecodeTopk) {
          topk_token<EPL>(row, LoadL2{}, p.E, p.k, lane, e, w);
        } else {
          SelectParams sp{row, p.bias, p.T, p.E, p.k, p.n_group, p.topk_group, p.renorm, p.scale, nullptr, nullptr};
          uint32_t* keys = s_keys + wr * (S::E + S::E / 32 + 1);
          const bool groups = p.n_group > 1;
          if (p.score == kDecodeSigmoid)
            groups ? select_token<EPL, false, true>(row, LoadL2{}, sp, keys, lane, e, w)
                   : select_token<EPL, false, false>(row, LoadL2{}, sp, keys, lane, e, w);
          else
            groups ? select_token<EPL, true, true>(row, LoadL2{}, sp, keys, lane, e, w)
                   : select_token<EPL, true, false>(row, LoadL2{}, sp, keys, lane, e, w);
        }
        if (lane < p.k) {
          s_idx[t * p.k + lane] = static_cast<uint16_t>(e);
          s_w[t * p.k + lane] = w;
          atomicOr(&s_mask[e], 1u << t);
          if (blockIdx.x == 0) {
            if (p.topk_idx != nullptr) p.topk_idx[t * p.k + lane] = e;
            if (p.topk_w != nullptr) p.topk_w[t * p.k + lane] = w;
          }
        }
      }
      bar_named(2, kRouteThreads);
      if (wr == 0) {
        // chosen experts ascending, each with its rows; lane l walks experts [l * EPL, +EPL)
        int rows = 0, chosen = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const uint32_t m = s_mask[lane * EPL + i];
          rows += __popc(m);
          chosen += m != 0u;
        }
        int row0 = rows, a0 = chosen;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int r = __shfl_up_sync(kFull, row0, d), a = __shfl_up_sync(kFull, a0, d);
          if (lane >= d) { row0 += r; a0 += a; }
        }
        const int all = __shfl_sync(kFull, a0, 31);
        row0 -= rows;
        a0 -= chosen;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          uint32_t m = s_mask[lane * EPL + i];
          if (m == 0u) continue;
          s_expert[a0] = static_cast<uint16_t>(lane * EPL + i);
          s_off[a0] = static_cast<uint16_t>(row0);
          ++a0;
          while (m != 0u) {
            s_token[row0++] = static_cast<uint8_t>(__ffs(m) - 1);
            m &= m - 1u;
          }
        }
        __syncwarp();
        if (lane == 0) {
          *s_chosen = all;
          s_off[all] = static_cast<uint16_t>(pairs);
        }
      }
      bar_named(2, kRouteThreads);
      for (int i = tid; i < pairs; i += kRouteThreads) {
        // the pair's row: its expert's first one and the earlier tokens that chose it
        const int t = i / p.k, e = s_idx[i];
        int lo = 0, hi = *s_chosen - 1;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (s_expert[mid] < e) lo = mid + 1; else hi = mid;
        }
        s_slot[i] = static_cast<uint16_t>(s_off[lo] + __popc(s_mask[e] & ((1u << t) - 1u)));
      }
      bar_named(2, kRouteThreads);
      if (tid == 0) mbar_arrive(plan_bar);
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

// [E][2F][K] bf16 (gate rows, then up rows) as (K, F rows, gate/up, E); a box holds 64 gate rows and the matching up rows.
int make_tmap_up(CUtensorMap* m, const void* base, long long K, long long F, long long E) {
  const unsigned long long dims[4] = {static_cast<unsigned long long>(K), static_cast<unsigned long long>(F), 2,
                                      static_cast<unsigned long long>(E)};
  const unsigned long long strides[3] = {2ull * K, 2ull * K * F, 4ull * K * F};
  const unsigned box[4] = {64, 64, 2, 1};
  return make_tmap_bf16(m, base, 4, dims, strides, box);
}

// [E][N][K] bf16 as (K, N rows, E); a box holds 128 rows.
int make_tmap_down(CUtensorMap* m, const void* base, long long K, long long N, long long E) {
  const unsigned long long dims[3] = {static_cast<unsigned long long>(K), static_cast<unsigned long long>(N),
                                      static_cast<unsigned long long>(E)};
  const unsigned long long strides[2] = {2ull * K, 2ull * K * N};
  const unsigned box[3] = {64, kUnitRows, 1};
  return make_tmap_bf16(m, base, 3, dims, strides, box);
}

// [rows][K] bf16 as (64, rows, K / 64): box_rows rows of `blocks` K blocks.
int make_tmap_rows(CUtensorMap* m, const void* base, long long K, long long rows, unsigned box_rows, unsigned blocks) {
  const unsigned long long dims[3] = {64, static_cast<unsigned long long>(rows), static_cast<unsigned long long>(K / 64)};
  const unsigned long long strides[2] = {2ull * K, 128};
  const unsigned box[3] = {64, box_rows, blocks};
  return make_tmap_bf16(m, base, 3, dims, strides, box);
}

int make_tmap_tokens(CUtensorMap* m, const void* base, long long K, long long rows) {
  const unsigned long long dims[2] = {static_cast<unsigned long long>(K), static_cast<unsigned long long>(rows)};
  const unsigned long long strides[1] = {2ull * K};
  const unsigned box[2] = {64, kTok};
  return make_tmap_bf16(m, base, 2, dims, strides, box);
}

template <int EPL>
int launch_decode(const DecodeCall& c, const DecodeParams& p, cudaStream_t st) {
  using S = DecodeShape<EPL>;
  DecodeMaps m{};
  int rc = make_tmap_rows(&m.router, c.w_router, p.H, p.E, kRouterRows, kRouterKb);
  if (!rc) rc = make_tmap_rows(&m.x_router, c.x, p.H, p.T, kTok, kRouterKb);
  if (!rc) rc = make_tmap_tokens(&m.x, c.x, p.H, p.T);
  if (!rc) rc = make_tmap_tokens(&m.h, p.h, p.F, p.T * p.k);
  if (!rc) rc = make_tmap_up(&m.w13, c.w13, p.H, p.F, p.E);
  if (!rc) rc = make_tmap_down(&m.w2, c.w2, p.F, p.H, p.E);
  if (!rc && p.Fs > 0) {
    rc = make_tmap_tokens(&m.hs, p.hs, p.Fs, p.T);
    if (!rc) rc = make_tmap_up(&m.ws13, c.ws13, p.H, p.Fs, 1);
    if (!rc) rc = make_tmap_down(&m.ws2, c.ws2, p.Fs, p.H, 1);
  }
  static std::atomic<uint64_t> attr_set{0};
  if (!rc) rc = set_smem_attr(reinterpret_cast<const void*>(moe_decode_kernel<EPL>), S::SMEM, attr_set);
  int sms = 0;
  if (!rc) rc = device_sm_count(&sms);
  if (rc) return rc;
  // as many blocks as the largest phase has units, one to an SM
  const long long experts = p.T * p.k < p.E ? p.T * p.k : p.E;
  const long long hb = (p.H + kUnitRows - 1) / kUnitRows;
  long long units = experts * (p.F / 64);
  if (experts * hb > units) units = experts * hb;
  const long long first = (p.E + kRouterRows - 1) / kRouterRows + p.Fs / 64;
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
  return p.E <= 256 ? launch_decode<8>(c, p, st) : launch_decode<16>(c, p, st);
}

}  // namespace invmoe
