// fp8_gemm.cu -- e4m3 matrix product with a scale per 1 x 128 of the tokens and 128 x 128 of the weights (sm_103a).
//
//   out[t, n] = sum_kb (as[t, kb] * ws[n / 128, kb]) * p_kb[t, n],   p_kb = sum_{k in block kb} a[t, k] * w[n, k]
//
// p_kb comes from the tensor cores (tcgen05 kind::f8f6f4, four K = 32 steps, fp32 in TMEM, a fresh accumulator for every
// block); its scale is an arbitrary fp32 number, so the sum over blocks cannot stay in TMEM: eight warps read each p_kb
// and keep acc = fma(p_kb, as * ws, acc) in fp32 registers, kb ascending.  No split of K, one order for every tile
// shape, and a column's chain depends on its own token only: the bits do not depend on the batch.
//
// Weights are the MMA's M side (128 rows = exactly one scale block of the weights, so ws is one number per sub-tile and
// block) and tokens its N side, in multiples of 16: a group of 20 tokens costs 32 columns, not 128 rows, and decode and
// prefill run the same kernel with another NT.
//   * one producer thread: per 128-byte K block one TMA box of 128 weight rows per sub-tile (MT of them) and one box of
//     NT token rows, 128-byte swizzle (the K-major operand layout; a block is one swizzle row);
//   * one MMA thread: 4 * MT MMAs per block into one of ACC TMEM buffers;
//   * two warpgroups, each with half of the token columns and all 128 lanes.  TMEM is read in the 16x256b shape: a
//     thread then holds 4 rows x NT/8 columns instead of one row x NT/2 columns, so it needs a quarter of the per-token
//     scales from shared memory (one row per thread would make those broadcast reads the bound).
// SwiGLU (MT = 2): sub-tile 0 holds 128 gate rows, sub-tile 1 the matching up rows; h = silu(g) * u, its absolute
// maximum over the 128 rows of the block, and e4m3(h / scale) leave the kernel, never g, u or an unquantised h.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "fp8.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace invmoe {

namespace {

enum Fp8Epi : int { FP8_F32 = 0, FP8_BF16 = 1, FP8_SWIGLU = 2 };

struct Fp8Params {
  const float* a_scale;     // [token rows, KB]
  const float* w_scale;     // [G][w_srows][KB]
  int KB;                   // blocks of 128 along K
  int N;                    // weight rows of one group that are outputs (SwiGLU: F)
  int w_group_rows;         // weight rows of one group (SwiGLU: 2F)
  int w_srows;              // rows of one group's scales
  int n_blocks;             // units along the weight rows
  int M;                    // token rows (dense)
  int G;                    // groups (0 = dense)
  const int* counts;
  const int* offsets;
  void* out;                // [token rows, N] fp32 / bf16 / e4m3
  float* out_scale;         // SwiGLU: [token rows, N / 128]
  int vec_scale;            // KB % 4 == 0 and 16-byte aligned bases: four blocks' scales in one load
  int vec_out;              // N % 4 == 0: outputs in vectors
  unsigned int* status;
  unsigned long long timeout_ns;
};

constexpr int kWTile = 128;                         // weight rows per sub-tile
constexpr int kWBytes = kWTile * kFp8Block;         // 16 KB
constexpr int kMaxGroups = 1024;
constexpr int kEpiWarps = 8;
constexpr int kScaleWarps = 2;
constexpr int kFirstEpiWarp = 2 + kScaleWarps;      // warp 0: producer, warp 1: MMA issuer, warps 2 and 3: scales
constexpr int kFp8Threads = 32 * (kFirstEpiWarp + kEpiWarps);
// Registers per thread: 168 at launch (65,536 / 384, whole units of 8).  A tile of 256 x 128 leaves 128 accumulators in
// each of the 256 epilogue threads, so there the first warpgroup hands registers over: 72 + 2 * 216 = 3 * 168.
constexpr int kLaunchRegs = 168, kLoaderRegs = 72, kEpiRegs = 216;
static_assert(kLoaderRegs + 2 * kEpiRegs <= 3 * kLaunchRegs, "register split");
constexpr int kStageF32 = kWTile + 4;               // floats per staged token row (conflict-free fragment writes)
constexpr int kStageFp8 = kWTile + 16;              // bytes per staged token row
constexpr int kStagingBytes = 9216;                 // per warpgroup: 16 x 132 floats or 64 x 144 bytes
static_assert(16 * kStageF32 * 4 <= kStagingBytes && 64 * kStageFp8 <= kStagingBytes, "staging");

template <int MT, int NT>
struct Fp8Shape {
  static constexpr int STAGE_BYTES = MT * kWBytes + NT * kFp8Block;
  static constexpr int ACC_COLS = MT * NT;
  static constexpr int ACC = 512 / ACC_COLS < 4 ? 512 / ACC_COLS : 4;   // TMEM buffers
  static constexpr int TMEM_COLS = ACC * ACC_COLS < 32 ? 32 : ACC * ACC_COLS;
  static constexpr int HALF = NT / 2;                                   // token columns of a warpgroup
  static constexpr int SLOT = NT + 4;                                   // a buffer's scales: NT tokens, MT weight blocks
  static constexpr int SCALE_BYTES = ACC * SLOT * 4;
  static constexpr int AMAX_BYTES = 2 * 4 * HALF * 4;                   // [warpgroup][warp][column]
  static constexpr int FIXED = 1024 + 2 * kStagingBytes + SCALE_BYTES + AMAX_BYTES + 256 + 4 * (kMaxGroups + 1) + 12;
  static constexpr int STAGES = (232448 - FIXED) / STAGE_BYTES < 8 ? (232448 - FIXED) / STAGE_BYTES : 8;
  static constexpr int SMEM_BYTES = FIXED + STAGES * STAGE_BYTES;
  static_assert(SMEM_BYTES <= 232448 && STAGES >= 3, "shared memory");
  static_assert(8 * (2 * STAGES + 2 * ACC) + 16 <= 256, "barriers");
};

// Instruction descriptor, kind::f8f6f4: e4m3 A and B (formats 0), fp32 D, both K-major.
__device__ __forceinline__ uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void umma_fp8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 16 TMEM lanes x 8 * X columns (16x256b shape): register 4i + {0, 1} holds lane t / 4, columns 8i + 2(t % 4) + {0, 1},
// register 4i + {2, 3} the same columns of lane t / 4 + 8 (t = lane of the warp).
template <int X>
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t taddr, uint32_t (&r)[4 * X]) {
  static_assert(X == 1 || X == 2 || X == 4 || X == 8, "repeat");
  if constexpr (X == 1) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
  } else if constexpr (X == 2) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  } else if constexpr (X == 4) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
  }
}

// The registers are seen as redefined here (after tcgen05.wait::ld), so no use of them moves above the wait.
template <int R>
__device__ __forceinline__ void reg_fence(uint32_t (&r)[R]) {
#pragma unroll
  for (int i = 0; i < R; ++i) asm volatile("" : "+r"(r[i]));
}

// Two fp32 fused multiply-adds, and two products, per instruction (each correctly rounded).
__device__ __forceinline__ void fma2(unsigned long long& acc, unsigned long long a, unsigned long long b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long pack2(uint32_t lo, uint32_t hi) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ float unpack2(unsigned long long v, int hi) {
  return __uint_as_float(static_cast<uint32_t>(hi ? v >> 32 : v));
}

// silu(g) * u.  The hardware's exponential and reciprocal: their few units in the last place vanish against the rounding
// to e4m3 that follows (2^-4), and the exact expf and division took a fifth of the gate/up kernel's time.  Both kernels
// use this expression, so h does not depend on which one runs.
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float swiglu(float g, float u) {
  return __fmul_rn(__fmul_rn(g, rcp_approx(__fadd_rn(1.0f, __expf(-g)))), u);
}

// All four warps of a warpgroup execute the one instruction of its side of the split.
__device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoaderRegs)); }
__device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs)); }

__device__ __forceinline__ void bar_wg(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

// mbar_wait by a whole warp, one answer for all lanes.
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, const WaitCtl& w) {
  if (__all_sync(0xffffffffu, mbar_test<CLUSTER>(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait_slow<CLUSTER>(bar, parity, w));
}

// Scales of blocks kb .. kb + 3 of one row (zeros past the last).
__device__ __forceinline__ float4 load_scales(const float* src, int kb, const Fp8Params& p) {
  if (p.vec_scale) return __ldg(reinterpret_cast<const float4*>(src + kb));
  float4 v = make_float4(__ldg(src + kb), 0.0f, 0.0f, 0.0f);
  if (kb + 1 < p.KB) v.y = __ldg(src + kb + 1);
  if (kb + 2 < p.KB) v.z = __ldg(src + kb + 2);
  if (kb + 3 < p.KB) v.w = __ldg(src + kb + 3);
  return v;
}

struct Fp8Unit {
  int row0;      // first token row
  int cols;      // tokens of this unit (1..NT)
  int g;         // group
  int nb;        // block of weight rows
};

// Units of a group: weight blocks outermost, token chunks innermost, so that the CTAs which share a weight tile run at
// about the same time and its second reader finds it in L2.
template <int NT>
__device__ __forceinline__ Fp8Unit fp8_unit(int u, const Fp8Params& p, const int* prefix, int total_chunks) {
  Fp8Unit U;
  if (p.G == 0) {
    U.g = 0;
    U.nb = u / total_chunks;
    const int c = u - U.nb * total_chunks;
    U.row0 = c * NT;
    U.cols = min(NT, p.M - U.row0);
    return U;
  }
  const int v = u / p.n_blocks;       // chunk index: group g owns [prefix[g], prefix[g + 1])
  int lo = 0, hi = p.G - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid + 1] > v) hi = mid;
    else lo = mid + 1;
  }
  U.g = lo;
  const int n_ch = prefix[lo + 1] - prefix[lo];
  const int r = u - prefix[lo] * p.n_blocks;
  U.nb = r / n_ch;
  const int c = r - U.nb * n_ch;
  U.row0 = __ldg(p.offsets + lo) + c * NT;
  U.cols = min(NT, __ldg(p.counts + lo) - c * NT);
  return U;
}

// One warp: prefix[g] = chunks of CH rows in the groups before g, and their total.
template <int CH>
__device__ __forceinline__ void prefix_chunks(const Fp8Params& p, int* prefix, int* total, int lane) {
  if (p.G == 0) {
    if (lane == 0) *total = (p.M + CH - 1) / CH;
    return;
  }
  const int per = (p.G + 31) / 32;
  const int g0 = lane * per;
  int local = 0;
  for (int i = 0; i < per; ++i)
    if (g0 + i < p.G) local += (__ldg(p.counts + g0 + i) + CH - 1) / CH;
  int incl = local;
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  int run = incl - local;
  for (int i = 0; i < per; ++i)
    if (g0 + i < p.G) {
      prefix[g0 + i] = run;
      run += (__ldg(p.counts + g0 + i) + CH - 1) / CH;
    }
  if (lane == 31) {
    prefix[p.G] = incl;
    *total = incl;
  }
}

template <int MT, int NT, int EPI>
__global__ void __launch_bounds__(kFp8Threads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
                    const Fp8Params p) {
  using S = Fp8Shape<MT, NT>;
  static_assert(EPI != FP8_SWIGLU || MT == 2, "SwiGLU pairs a gate sub-tile with its up sub-tile");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = ring + S::STAGES * S::STAGE_BYTES;
  float* s_scale = reinterpret_cast<float*>(staging + 2 * kStagingBytes);
  float* s_amax = s_scale + S::SCALE_BYTES / 4;
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(s_amax) + S::AMAX_BYTES);
  uint64_t* empty_bar = full_bar + S::STAGES;
  uint64_t* accf_bar = empty_bar + S::STAGES;
  uint64_t* acce_bar = accf_bar + S::ACC;
  uint32_t* misc = reinterpret_cast<uint32_t*>(acce_bar + S::ACC);
  uint32_t* tmem_slot = misc;
  volatile int* s_abort = reinterpret_cast<volatile int*>(misc + 1);
  int* s_total = reinterpret_cast<int*>(misc + 2);
  int* s_prefix = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(full_bar) + 256);   // [G + 1]

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int a = 0; a < S::ACC; ++a) {
      mbar_init(&accf_bar[a], 1 + kScaleWarps);
      mbar_init(&acce_bar[a], kEpiWarps);
    }
    *s_abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmA);
  }
  if (warp == 1) tmem_alloc(tmem_slot, S::TMEM_COLS);
  // everything above touches only shared memory, TMEM and the kernel parameters
  pdl_wait();
  pdl_trigger();
  if (warp == 2) prefix_chunks<NT>(p, s_prefix, s_total, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem_base = *tmem_slot;
  const int total_chunks = *s_total;
  const int total_units = total_chunks * p.n_blocks;
  WaitCtl wc{s_abort, p.status, p.timeout_ns};

  constexpr bool SPLIT_REGS = MT * NT >= 256;
  if (warp < kFirstEpiWarp) {
    if constexpr (SPLIT_REGS) give_registers();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- producer
      int stage = 0;
      uint32_t phase = 0;
      int fills = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < total_units; u += gridDim.x) {
        const Fp8Unit U = fp8_unit<NT>(u, p, s_prefix, total_chunks);
        int wrow[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m)
          wrow[m] = EPI == FP8_SWIGLU ? U.g * p.w_group_rows + m * p.N + U.nb * kWTile
                                      : U.g * p.w_group_rows + (U.nb * MT + m) * kWTile;
        for (int kb = 0; kb < p.KB; ++kb) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1u, wc)) { ok = false; break; }
          uint8_t* st = ring + stage * S::STAGE_BYTES;
          mbar_arrive_expect_tx(&full_bar[stage], S::STAGE_BYTES);   // a box counts its full size, filled rows included
#pragma unroll
          for (int m = 0; m < MT; ++m) tma_load_2d(st + m * kWBytes, &tmW, &full_bar[stage], kb * kFp8Block, wrow[m]);
          tma_load_2d(st + MT * kWBytes, &tmA, &full_bar[stage], kb * kFp8Block, U.row0);
          ++fills;
          if (++stage == S::STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // every copy this thread issued lands before the CTA can exit
      WaitCtl drain{nullptr, p.status, p.timeout_ns};
      for (int s = 0; s < S::STAGES && s < fills; ++s)   // the last of this stage's fills
        mbar_wait(&full_bar[s], static_cast<uint32_t>((fills - 1 - s) / S::STAGES) & 1u, drain);
    } else if (warp == 1 && lane == 0) {
      // ---------------------------------------------------------- MMA issuer
      const uint64_t wdesc0 = sdesc_k_sw128(smem_u32(ring));
      const uint64_t adesc0 = sdesc_k_sw128(smem_u32(ring + MT * kWBytes));
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      bool issued = false;
      int last_acc = 0;
      uint32_t last_phase = 0;
      for (int u = blockIdx.x; ok && u < total_units; u += gridDim.x) {
        const Fp8Unit U = fp8_unit<NT>(u, p, s_prefix, total_chunks);
        const uint32_t idesc = idesc_e4m3_f32(kWTile, (U.cols + 15) & ~15);
        for (int kb = 0; kb < p.KB; ++kb) {
          if (!mbar_wait(&acce_bar[acc], acc_phase ^ 1u, wc) || !mbar_wait(&full_bar[stage], phase, wc)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t so = static_cast<uint64_t>((stage * S::STAGE_BYTES) >> 4);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const uint32_t d = tmem_base + static_cast<uint32_t>(acc * S::ACC_COLS + m * NT);
#pragma unroll
            for (int kk = 0; kk < kFp8Block / 32; ++kk)   // K = 32 steps: 32 bytes on inside the swizzle row
              umma_fp8(d, wdesc0 + so + static_cast<uint64_t>(m * (kWBytes >> 4)) + 2u * kk, adesc0 + so + 2u * kk, idesc,
                       kk != 0 ? 1u : 0u);
          }
          umma_commit(&empty_bar[stage]);
          umma_commit(&accf_bar[acc]);
          issued = true;
          last_acc = acc;
          last_phase = acc_phase;
          if (++stage == S::STAGES) { stage = 0; phase ^= 1u; }
          if (++acc == S::ACC) { acc = 0; acc_phase ^= 1u; }
        }
      }
      if (!ok) *s_abort = 1;
      // every MMA issued here has finished before the CTA releases TMEM
      WaitCtl drain{nullptr, p.status, p.timeout_ns};
      if (issued) mbar_wait(&accf_bar[last_acc], last_phase, drain);
    } else if (warp >= 2) {
      // ---------------------------------------------------------- scales
      // Thread j prepares the scales of tokens j and j + 64 for every block, as they are needed: buffer `acc` gets them
      // together with its products (its barrier counts the MMA's commit and these two warps).  Four blocks' scales
      // come in one load (or four), issued four blocks ahead.
      constexpr int PER = NT > 64 ? NT / 64 : 1;
      const int j0 = (warp - 2) * 32 + lane;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < total_units; u += gridDim.x) {
        const Fp8Unit U = fp8_unit<NT>(u, p, s_prefix, total_chunks);
        // PER token rows, then (threads below MT) a weight block row
        const float* src[PER + 1];
        bool on[PER + 1];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int c = j0 + 64 * i;
          src[i] = p.a_scale + static_cast<long long>(U.row0 + min(c, U.cols - 1)) * p.KB;
          on[i] = c < NT;
        }
        {
          const int srow = EPI == FP8_SWIGLU ? j0 * (p.N / kFp8Block) + U.nb : U.nb * MT + j0;
          src[PER] = p.w_scale + (static_cast<long long>(U.g) * p.w_srows + min(srow, p.w_srows - 1)) * p.KB;
          on[PER] = j0 < MT;
        }
        float4 next[PER + 1];
#pragma unroll
        for (int i = 0; i <= PER; ++i) next[i] = on[i] ? load_scales(src[i], 0, p) : make_float4(0.f, 0.f, 0.f, 0.f);
        for (int kb0 = 0; ok && kb0 < p.KB; kb0 += 4) {
          float4 cur[PER + 1];
#pragma unroll
          for (int i = 0; i <= PER; ++i) {
            cur[i] = next[i];
            if (on[i] && kb0 + 4 < p.KB) next[i] = load_scales(src[i], kb0 + 4, p);
          }
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            if (kb0 + d >= p.KB) break;
            ok = __all_sync(0xffffffffu, mbar_wait(&acce_bar[acc], acc_phase ^ 1u, wc));
            if (!ok) break;
            float* slot = s_scale + acc * S::SLOT;
#pragma unroll
            for (int i = 0; i <= PER; ++i)
              if (on[i]) {
                const float v = d == 0 ? cur[i].x : d == 1 ? cur[i].y : d == 2 ? cur[i].z : cur[i].w;
                slot[i < PER ? j0 + 64 * i : NT + j0] = v;
              }
            __syncwarp();
            if (lane == 0) mbar_arrive(&accf_bar[acc]);
            if (++acc == S::ACC) { acc = 0; acc_phase ^= 1u; }
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ scaling and epilogue
    if constexpr (SPLIT_REGS) take_registers();
    // All eight warps walk the same units whatever happens, so the warpgroup barriers always meet; after a
    // wait that ran out (ok = false) a warp only keeps those barriers.
    constexpr int X = NT / 16;                         // 8-column fragments of a warpgroup's columns
    const int q = warp & 3;                            // TMEM lane quadrant
    const int half = (warp - kFirstEpiWarp) >> 2;                  // warpgroup: token columns [half * HALF, +HALF)
    const int tid = q * 32 + lane;                     // thread of the warpgroup
    const int bar_id = 1 + half;
    float* my_amax = s_amax + half * (4 * S::HALF);
    uint8_t* stg = staging + half * kStagingBytes;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < total_units; u += gridDim.x) {
      const Fp8Unit U = fp8_unit<NT>(u, p, s_prefix, total_chunks);
      const int wg_cols = U.cols - half * S::HALF;     // this warpgroup's tokens (may be <= 0)
      // accumulators in pairs of neighbouring columns: [sub-tile][16-lane half][fragment, row of 8]
      unsigned long long v2[MT][2][2 * X];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 2 * X; ++i) v2[m][h][i] = 0ull;
      for (int kb = 0; kb < p.KB; ++kb) {
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait_inline(&accf_bar[acc], acc_phase, wc));
        if (ok) {
          tc_fence_after();
          if (wg_cols > 0) {
            const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                static_cast<uint32_t>(acc * S::ACC_COLS + half * S::HALF);
            const float* slot = s_scale + acc * S::SLOT;
            unsigned long long wsc[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              const uint32_t w = __float_as_uint(slot[NT + m]);
              wsc[m] = pack2(w, w);
            }
            // steps of XC fragments of one sub-tile, both 16-lane halves; the next step's TMEM loads are in flight
            // while this step's products are added
            constexpr int XC = X < 4 ? X : 4;
            constexpr int STEPS = X / XC * MT;
            uint32_t r[2][2][4 * XC];
            unsigned long long asc[XC];
            auto issue = [&](int st) {
              const uint32_t at = tb + static_cast<uint32_t>((st % MT) * NT + (st / MT) * XC * 8);
              tmem_ld_16x256b<XC>(at, r[st & 1][0]);
              tmem_ld_16x256b<XC>(at + (16u << 16), r[st & 1][1]);
            };
            issue(0);
#pragma unroll
            for (int st = 0; st < STEPS; ++st) {
              const int m = st % MT, c = st / MT;
              if (m == 0) {
#pragma unroll
                for (int i = 0; i < XC; ++i)
                  asc[i] = *reinterpret_cast<const unsigned long long*>(slot + half * S::HALF + 8 * (c * XC + i) +
                                                                        2 * (lane & 3));
              }
              tmem_ld_wait();
              reg_fence(r[st & 1][0]);
              reg_fence(r[st & 1][1]);
              if (st + 1 < STEPS) issue(st + 1);
#pragma unroll
              for (int i = 0; i < XC; ++i) {
                const unsigned long long sc = mul2(asc[i], wsc[m]);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    fma2(v2[m][h][2 * (c * XC + i) + e],
                         pack2(r[st & 1][h][4 * i + 2 * e], r[st & 1][h][4 * i + 2 * e + 1]), sc);
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acce_bar[acc]);
        }
        if (++acc == S::ACC) { acc = 0; acc_phase ^= 1u; }
      }
      float v[MT][2][4 * X];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4 * X; ++i) v[m][h][i] = unpack2(v2[m][h][i >> 1], i & 1);
      const long long out_row0 = static_cast<long long>(U.row0) + half * S::HALF;
      if constexpr (EPI == FP8_SWIGLU) {
        bar_wg(bar_id);                                // the previous unit's maxima and staging have been read
        // h in place of the gate values; each column's absolute maximum over the thread's 4 rows, the warp's 32
        // (lanes that differ in lane / 4) and the 4 warps
#pragma unroll
        for (int i = 0; i < X; ++i) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float mx = 0.0f;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float& g = v[0][h][4 * i + j + 2 * e];
                g = swiglu(g, v[1][h][4 * i + j + 2 * e]);
                mx = fmaxf(mx, fabsf(g));
              }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            if (lane < 4) my_amax[q * S::HALF + 8 * i + 2 * lane + j] = mx;
          }
        }
        bar_wg(bar_id);
        float my_s = 0.0f;
        if (tid < S::HALF) {
          const float a = fmaxf(fmaxf(my_amax[tid], my_amax[S::HALF + tid]),
                                fmaxf(my_amax[2 * S::HALF + tid], my_amax[3 * S::HALF + tid]));
          my_s = fp8_scale(a);
        }
        bar_wg(bar_id);
        if (tid < S::HALF) {
          my_amax[tid] = __frcp_rn(my_s);
          if (ok && tid < wg_cols) p.out_scale[(out_row0 + tid) * (p.N / kFp8Block) + U.nb] = my_s;
        }
        bar_wg(bar_id);
#pragma unroll
        for (int i = 0; i < X; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int col = 8 * i + 2 * (lane & 3) + j;
            const float inv = my_amax[col];
            uint8_t* d = stg + col * kStageFp8 + q * 32 + (lane >> 2);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 2; ++e) d[16 * h + 8 * e] = fp8_one(v[0][h][4 * i + j + 2 * e], inv);
          }
        bar_wg(bar_id);
        // 8 lanes of 16 bytes per token row
        uint8_t* out = static_cast<uint8_t*>(p.out) + out_row0 * p.N + static_cast<long long>(U.nb) * kWTile;
        for (int t = tid >> 3; t < S::HALF; t += 16)
          if (ok && t < wg_cols)
            *reinterpret_cast<uint4*>(out + static_cast<long long>(t) * p.N + 16 * (tid & 7)) =
                *reinterpret_cast<const uint4*>(stg + t * kStageFp8 + 16 * (tid & 7));
      } else {
        constexpr int CI = X < 2 ? 1 : 2;              // fragments (8 tokens each) staged at a time
        float* stf = reinterpret_cast<float*>(stg);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int n0 = (U.nb * MT + m) * kWTile;
#pragma unroll
          for (int i0 = 0; i0 < X; i0 += CI) {
            bar_wg(bar_id);
#pragma unroll
            for (int ii = 0; ii < CI; ++ii)
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  stf[(8 * ii + 2 * (lane & 3) + (e & 1)) * kStageF32 + q * 32 + 16 * h + 8 * (e >> 1) + (lane >> 2)] =
                      v[m][h][4 * (i0 + ii) + e];
            bar_wg(bar_id);
            // one warp per token row: 4 outputs per lane
#pragma unroll
            for (int tt = q; tt < 8 * CI; tt += 4) {
              const int t = 8 * i0 + tt;
              const int n = n0 + 4 * lane;
              if (!ok || t >= wg_cols || n >= p.N) continue;
              const float4 o = *reinterpret_cast<const float4*>(stf + tt * kStageF32 + 4 * lane);
              const long long at = (out_row0 + t) * p.N + n;
              if constexpr (EPI == FP8_F32) {
                float* d = static_cast<float*>(p.out) + at;
                if (p.vec_out) {
                  *reinterpret_cast<float4*>(d) = o;
                } else {
                  d[0] = o.x;
                  if (n + 1 < p.N) d[1] = o.y;
                  if (n + 2 < p.N) d[2] = o.z;
                  if (n + 3 < p.N) d[3] = o.w;
                }
              } else {
                __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.out) + at;
                if (p.vec_out) {
                  const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
                  *reinterpret_cast<uint2*>(d) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                            *reinterpret_cast<const uint32_t*>(&hi));
                } else {
                  d[0] = __float2bfloat16_rn(o.x);
                  if (n + 1 < p.N) d[1] = __float2bfloat16_rn(o.y);
                  if (n + 2 < p.N) d[2] = __float2bfloat16_rn(o.z);
                  if (n + 3 < p.N) d[3] = __float2bfloat16_rn(o.w);
                }
              }
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, S::TMEM_COLS);
  }
}

// ------------------------------------------------------------ many rows: tokens on the M side
//
// The same product with the roles exchanged: a CTA computes 128 token rows x 256 weight rows (one N = 256 MMA per K = 32
// step).  A thread holds one token row, so its scale is one number per block, read from global memory four blocks ahead:
// no shared memory on the scaling path, where the kernel above reads a scale for every column.
// What bounds it is neither the loads nor the tensor cores (without the scaling 8192 x 4096 x 6144 takes 129 us) but the
// handover of the products: 128 x 256 fp32 per block through TMEM and 256 FFMA issue cycles per scheduler, with two TMEM
// buffers to hide a commit, a wait and a release behind.  So a buffer is released as soon as its last columns are in
// registers, and the issuing warp runs converged (see umma_fp8_if).
// Measured and not kept (8192 x 4096 x 6144, 191 us): CTA pairs with 256 x 256 tiles, 183 us, but 663 instead of 549 us
// for 64 experts of about 256 rows, because the tiles are twice as high; four buffers of 128 columns, 260 us (an N = 128
// MMA takes more than half the time of an N = 256 one); packed fma.rn.f32x2, 690 instead of 485 cycles a block.
// SwiGLU: the 256 weight rows are 128 gate rows and the matching up rows.  A warpgroup has columns 64 half .. + 63 of
// either 128, so that a thread holds gate and up of the same h.
struct Fp8RowsShape {
  static constexpr int TILE_BYTES = kWTile * kFp8Block;       // 16 KB: 128 rows x 128 e4m3
  static constexpr int STAGE_BYTES = 3 * TILE_BYTES;          // token rows, then two tiles of weight rows
  static constexpr int STAGES = 4;
  static constexpr int ACC_COLS = 256;
  static constexpr int ACC = 2;                               // TMEM buffers
  static constexpr int OSTAGE_BYTES = kEpiWarps * 32 * 64;
  static constexpr int AMAX_BYTES = 2 * 2 * kWTile * 4;       // [unit parity][warpgroup][row]
  static constexpr int BAR_BYTES = 256;
  static constexpr int SMEM_BYTES =
      1024 + STAGES * STAGE_BYTES + OSTAGE_BYTES + AMAX_BYTES + BAR_BYTES + 4 * (kMaxGroups + 1) + 12;
  static_assert(SMEM_BYTES <= 232448, "shared memory");
  static_assert(8 * (2 * STAGES + 2 * ACC + 1) + 16 <= BAR_BYTES, "barriers");
};

// The MMA is predicated, not branched around: in converged code the descriptors stay in uniform registers, where the
// instruction wants them; issued from a branch of one lane each MMA cost some 140 cycles of moves.
__device__ __forceinline__ void umma_fp8_if(uint32_t on, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                 uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}

// umma_commit of the lane whose `on` is set.
__device__ __forceinline__ void umma_commit_if(uint32_t on, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(on)
      : "memory");
}

// A warp's 32 rows x 16 * PIECES bytes from registers (one row per lane) to global memory, whole rows of 64 or 128 bytes
// at a time (PIECES lanes per row), through 2 KB of shared memory: 32 rows of 64 bytes, or twice 16 rows of 128.  The
// 16-byte piece c of row r sits at piece c ^ (r / 2 or r) of its row, free of bank conflicts both ways.  Rows whose
// length is not a multiple of 16 bytes are written element by element.
template <int ELT, int PIECES>
__device__ __forceinline__ void store_rows(uint8_t* stage, const uint32_t (&v)[4 * PIECES], uint8_t* out,
                                           long long ld_bytes, int rows_valid, long long bytes_valid, bool vec) {
  static_assert(PIECES == 4 || PIECES == 8, "64 or 128 bytes");
  constexpr int ROWS = 128 / PIECES;                   // rows staged at a time
  const int lane = threadIdx.x & 31;
  auto at = [&](int r, int c) { return stage + r * (16 * PIECES) + ((c ^ (PIECES == 8 ? r & 7 : (r >> 1) & 3)) << 4); };
  const int c = lane % PIECES;
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += ROWS) {
    if (lane >= r0 && lane < r0 + ROWS) {
#pragma unroll
      for (int k = 0; k < PIECES; ++k)
        *reinterpret_cast<uint4*>(at(lane - r0, k)) = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * (32 / PIECES) + lane / PIECES;
      const uint4 w = *reinterpret_cast<const uint4*>(at(r, c));
      if (r0 + r < rows_valid && c * 16 < bytes_valid) {
        uint8_t* d = out + (r0 + r) * ld_bytes + c * 16;
        if (vec) {
          *reinterpret_cast<uint4*>(d) = w;
        } else {
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 16 / ELT; ++e) {
            if (c * 16 + e * ELT < bytes_valid) {
              if (ELT == 4) *reinterpret_cast<uint32_t*>(d + 4 * e) = x[e];
              else *reinterpret_cast<uint16_t*>(d + 2 * e) = static_cast<uint16_t>(x[e >> 1] >> (16 * (e & 1)));
            }
          }
        }
      }
    }
    __syncwarp();
  }
}

template <int EPI>
__global__ void __launch_bounds__(kFp8Threads, 1)
    fp8_rows_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
                    const Fp8Params p) {
  using S = Fp8RowsShape;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ostage = ring + S::STAGES * S::STAGE_BYTES;
  float* s_amax = reinterpret_cast<float*>(ostage + S::OSTAGE_BYTES);
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(s_amax) + S::AMAX_BYTES);
  uint64_t* empty_bar = full_bar + S::STAGES;
  uint64_t* accf_bar = empty_bar + S::STAGES;
  uint64_t* acce_bar = accf_bar + S::ACC;
  uint64_t* final_bar = acce_bar + S::ACC;
  uint32_t* misc = reinterpret_cast<uint32_t*>(final_bar + 1);
  uint32_t* tmem_slot = misc;
  volatile int* s_abort = reinterpret_cast<volatile int*>(misc + 1);
  int* s_total = reinterpret_cast<int*>(misc + 2);
  int* s_prefix = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(full_bar) + S::BAR_BYTES);   // [G + 1]

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  constexpr int CH = kWTile;                        // token rows of a unit

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int a = 0; a < S::ACC; ++a) {
      mbar_init(&accf_bar[a], 1);
      mbar_init(&acce_bar[a], kEpiWarps);
    }
    mbar_init(final_bar, 1);
    *s_abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmA);
  }
  if (warp == 1) tmem_alloc(tmem_slot, S::ACC * S::ACC_COLS);
  // everything above touches only shared memory, TMEM and the kernel parameters
  pdl_wait();
  pdl_trigger();
  if (warp == 2) prefix_chunks<CH>(p, s_prefix, s_total, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem_base = *tmem_slot;
  const int total_chunks = *s_total;
  const int total_units = total_chunks * p.n_blocks;
  WaitCtl wc{s_abort, p.status, p.timeout_ns};

  if (warp < kFirstEpiWarp) {
    give_registers();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- producer
      int stage = 0;
      uint32_t phase = 0;
      int fills = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < total_units; u += gridDim.x) {
        const Fp8Unit U = fp8_unit<CH>(u, p, s_prefix, total_chunks);
        const int w_row = U.g * p.w_group_rows + (EPI == FP8_SWIGLU ? 1 : 2) * U.nb * kWTile;
        const int w_row1 = EPI == FP8_SWIGLU ? w_row + p.N : w_row + kWTile;
        for (int kb = 0; kb < p.KB; ++kb) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1u, wc)) { ok = false; break; }
          uint8_t* st = ring + stage * S::STAGE_BYTES;
          mbar_arrive_expect_tx(&full_bar[stage], S::STAGE_BYTES);
          tma_load_2d(st, &tmA, &full_bar[stage], kb * kFp8Block, U.row0);
          tma_load_2d(st + S::TILE_BYTES, &tmW, &full_bar[stage], kb * kFp8Block, w_row);
          tma_load_2d(st + 2 * S::TILE_BYTES, &tmW, &full_bar[stage], kb * kFp8Block, w_row1);
          ++fills;
          if (++stage == S::STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // every copy this thread issued lands before the CTA can exit
      WaitCtl drain{nullptr, p.status, p.timeout_ns};
      for (int s = 0; s < S::STAGES && s < fills; ++s)   // the last of this stage's fills
        mbar_wait(&full_bar[s], static_cast<uint32_t>((fills - 1 - s) / S::STAGES) & 1u, drain);
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer: the whole warp, one lane issues
      const uint32_t on = lane == 0 ? 1u : 0u;
      const uint64_t adesc0 = sdesc_k_sw128(smem_u32(ring));
      const uint64_t wdesc0 = sdesc_k_sw128(smem_u32(ring + S::TILE_BYTES));
      const uint32_t idesc = idesc_e4m3_f32(kWTile, S::ACC_COLS);
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < total_units; u += gridDim.x) {
        for (int kb = 0; kb < p.KB; ++kb) {
          if (!wait_warp(&acce_bar[acc], acc_phase ^ 1u, wc) || !wait_warp(&full_bar[stage], phase, wc)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t so = static_cast<uint64_t>((stage * S::STAGE_BYTES) >> 4);
          const uint32_t d = tmem_base + static_cast<uint32_t>(acc * S::ACC_COLS);
#pragma unroll
          for (int kk = 0; kk < kFp8Block / 32; ++kk)
            umma_fp8_if(on, d, adesc0 + so + 2u * kk, wdesc0 + so + 2u * kk, idesc, kk != 0 ? 1u : 0u);
          umma_commit_if(on, &accf_bar[acc]);
          umma_commit_if(on, &empty_bar[stage]);
          if (++stage == S::STAGES) { stage = 0; phase ^= 1u; }
          if (++acc == S::ACC) { acc = 0; acc_phase ^= 1u; }
        }
      }
      if (!ok) *s_abort = 1;
      // every MMA issued here has finished before the CTA releases TMEM
      if (lane == 0) umma_commit(final_bar);
      WaitCtl drain{nullptr, p.status, p.timeout_ns};
      mbar_wait(final_bar, 0, drain);
    }
  } else {
    // ------------------------------------------------------------ scaling and epilogue
    // All eight warps walk the same units whatever happens, so the SwiGLU barrier always meets; after a wait that ran
    // out (ok = false) a warp only keeps that barrier.
    take_registers();
    const int q = warp & 3;                            // TMEM lane quadrant
    const int ew = warp - kFirstEpiWarp;
    const int half = ew >> 2;                          // warpgroup: weight rows 64 half .. + 63 of either CTA's 128
    const int r_in_tile = q * 32 + lane;
    
    uint8_t* stg = ostage + ew * 32 * 64;
    int acc = 0;
    uint32_t acc_phase = 0;
    int parity = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < total_units; u += gridDim.x) {
      const Fp8Unit U = fp8_unit<CH>(u, p, s_prefix, total_chunks);
      const int first = q * 32;                        // the warp's first row of the unit
      const int rows_valid = U.cols - first;           // may be <= 0: nothing to scale or store
      const float* ap = p.a_scale + static_cast<long long>(U.row0 + min(first + lane, U.cols - 1)) * p.KB;
      // weight scales of the two blocks of 128 weight rows (SwiGLU: gate and up)
      const float* wbase = p.w_scale + static_cast<long long>(U.g) * p.w_srows * p.KB;
      const int sr0 = EPI == FP8_SWIGLU ? U.nb : 2 * U.nb;
      const int sr1 = EPI == FP8_SWIGLU ? U.nb + p.N / kFp8Block : min(2 * U.nb + 1, p.w_srows - 1);
      const float* wp0 = wbase + static_cast<long long>(sr0) * p.KB;
      const float* wp1 = wbase + static_cast<long long>(sr1) * p.KB;
      float v[4][32];                                  // 64 columns of the first 128 weight rows, then 64 of the second
#pragma unroll
      for (int st = 0; st < 4; ++st)
#pragma unroll
        for (int i = 0; i < 32; ++i) v[st][i] = 0.0f;
      float4 an = load_scales(ap, 0, p), wn0 = load_scales(wp0, 0, p), wn1 = load_scales(wp1, 0, p);
      for (int kb0 = 0; kb0 < p.KB; kb0 += 4) {
        float4 ac = an, wc0 = wn0, wc1 = wn1;
        if (kb0 + 4 < p.KB) {
          an = load_scales(ap, kb0 + 4, p);
          wn0 = load_scales(wp0, kb0 + 4, p);
          wn1 = load_scales(wp1, kb0 + 4, p);
        }
        const int n_kb = min(4, p.KB - kb0);
        // not unrolled (that measured slower): the scales of the next block move up instead
#pragma unroll 1
        for (int d = 0; d < n_kb; ++d) {
          const float s0 = __fmul_rn(ac.x, wc0.x), s1 = __fmul_rn(ac.x, wc1.x);
          ac.x = ac.y; ac.y = ac.z; ac.z = ac.w;
          wc0.x = wc0.y; wc0.y = wc0.z; wc0.z = wc0.w;
          wc1.x = wc1.y; wc1.y = wc1.z; wc1.z = wc1.w;
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait_inline(&accf_bar[acc], acc_phase, wc));
          if (ok) {
            tc_fence_after();
            if (rows_valid > 0) {
              const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                  static_cast<uint32_t>(acc * S::ACC_COLS + half * 64);
              uint32_t r[2][32];
              tmem_ld32(tb, r[0]);
#pragma unroll
              for (int st = 0; st < 4; ++st) {
                tmem_ld_wait();
                tmem_reg_fence(r[st & 1]);
                if (st < 3) {
                  tmem_ld32(tb + 32 * ((st + 1) & 1) + kWTile * ((st + 1) >> 1), r[(st + 1) & 1]);
                } else {
                  // everything is in registers: the buffer is free before the last products are added
                  tc_fence_before();
                  __syncwarp();
                  if (lane == 0) mbar_arrive(&acce_bar[acc]);
                }
                const float sc = st < 2 ? s0 : s1;
                // one FFMA per product: pairs in fma.rn.f32x2 measured slower here (485 -> 690 cycles a block)
#pragma unroll
                for (int i = 0; i < 32; ++i) v[st][i] = fmaf(__uint_as_float(r[st & 1][i]), sc, v[st][i]);
              }
            } else if (lane == 0) {
              mbar_arrive(&acce_bar[acc]);
            }
          }
          if (++acc == S::ACC) { acc = 0; acc_phase ^= 1u; }
        }
      }
      const long long row0 = static_cast<long long>(U.row0) + first;
      if constexpr (EPI == FP8_SWIGLU) {
        float h[64];
        float mx = 0.0f;
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          const float g = v[i >> 5][i & 31], up = v[2 + (i >> 5)][i & 31];
          h[i] = swiglu(g, up);
          mx = fmaxf(mx, fabsf(h[i]));
        }
        float* am = s_amax + parity * 2 * kWTile;
        am[half * kWTile + r_in_tile] = mx;
        // two buffers by unit parity: a buffer is written again only after the next unit's barrier
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const float sc = fp8_scale(fmaxf(am[r_in_tile], am[kWTile + r_in_tile]));
        parity ^= 1;
        if (ok && rows_valid > 0) {
          const float inv = __frcp_rn(sc);
          uint32_t packed[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) packed[i] = fp8_pack4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3], inv);
          if (half == 0 && lane < rows_valid) p.out_scale[(row0 + lane) * (p.N / kFp8Block) + U.nb] = sc;
          store_rows<4, 4>(stg, packed, static_cast<uint8_t*>(p.out) + row0 * p.N + U.nb * kWTile + half * 64, p.N,
                           rows_valid, 64, true);
        }
      } else if (ok && rows_valid > 0) {
        constexpr int ELT = EPI == FP8_F32 ? 4 : 2;
        const long long ld = static_cast<long long>(p.N) * ELT;
        // fp32: 32 columns, bf16: 64 columns to a row of 128 bytes
        constexpr int COLS = 128 / ELT;
#pragma unroll
        for (int part = 0; part < 128 / COLS; ++part) {
          const int n = (2 * U.nb + part * COLS / 64) * kWTile + half * 64 + part * COLS % 64;
          if (n >= p.N) continue;
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if constexpr (EPI == FP8_F32) {
              w[i] = __float_as_uint(v[part][i]);
            } else {
              const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * part + (i >> 4)][2 * (i & 15)],
                                                             v[2 * part + (i >> 4)][2 * (i & 15) + 1]);
              w[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
          }
          store_rows<ELT, 8>(stg, w, static_cast<uint8_t*>(p.out) + row0 * ld + static_cast<long long>(n) * ELT, ld,
                             rows_valid, static_cast<long long>(p.N - n) * ELT, p.vec_out != 0);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, S::ACC * S::ACC_COLS);
  }
}

// The register split must not ask for more than the launch holds: a kernel that waits for registers never ends.
int check_launch_regs(const void* kernel, const char* name, std::atomic<int>& regs) {
  int r = regs.load(std::memory_order_relaxed);
  if (r == 0) {
    cudaFuncAttributes fa;
    const int rc = check_cuda(cudaFuncGetAttributes(&fa, kernel), "cudaFuncGetAttributes");
    if (rc) return rc;
    r = fa.numRegs;
    regs.store(r, std::memory_order_relaxed);
  }
  if (r != kLaunchRegs) return set_error(INVMOE_ERR_CUDA, "%s: compiled with %d registers, not %d", name, r, kLaunchRegs);
  return INVMOE_OK;
}

int check_units(const Fp8Call& c, int chunk, int n_blocks, long long* units) {
  const long long chunks = c.G > 0 ? static_cast<long long>(c.rows) / chunk + (c.rows < c.G ? c.rows : c.G)
                                   : (static_cast<long long>(c.rows) + chunk - 1) / chunk;
  *units = chunks * n_blocks;
  if (*units > 0x7fffffffLL) return set_error(INVMOE_ERR_UNSUPPORTED_SHAPE, "%s: too many tiles for one launch", c.name);
  return INVMOE_OK;
}

int make_maps(const Fp8Call& c, const Fp8Params& p, int token_box, CUtensorMap* w, CUtensorMap* a) {
  const int rc = make_tmap_fp8(w, c.w, c.K, static_cast<long long>(p.w_group_rows) * (c.G > 0 ? c.G : 1), kWTile);
  return rc ? rc : make_tmap_fp8(a, c.a, c.K, c.rows, token_box);
}

template <int EPI>
int launch_rows(const Fp8Call& c, Fp8Params p, cudaStream_t st) {
  using S = Fp8RowsShape;
  const void* kernel = reinterpret_cast<const void*>(fp8_rows_kernel<EPI>);
  p.n_blocks = EPI == FP8_SWIGLU ? c.N / kWTile : (c.N + 2 * kWTile - 1) / (2 * kWTile);
  p.vec_out = static_cast<long long>(c.N) * (EPI == FP8_F32 ? 4 : 2) % 16 == 0;
  long long units = 0;
  int rc = check_units(c, kWTile, p.n_blocks, &units);
  CUtensorMap tmW, tmA;
  if (rc == INVMOE_OK) rc = make_maps(c, p, kWTile, &tmW, &tmA);
  static std::atomic<uint64_t> attr_set{0};
  static std::atomic<int> regs{0};
  if (rc == INVMOE_OK) rc = set_smem_attr(kernel, S::SMEM_BYTES, attr_set);
  if (rc == INVMOE_OK) rc = check_launch_regs(kernel, c.name, regs);
  int sms = 0;
  if (rc == INVMOE_OK) rc = device_sm_count(&sms);
  if (rc) return rc;
    const unsigned grid = static_cast<unsigned>(units < sms ? units : sms);
  ProfScope prof(c.name, st);
  return check_cuda(launch_kernel(fp8_rows_kernel<EPI>, dim3(grid), dim3(kFp8Threads), S::SMEM_BYTES, st,
                                     tmW, tmA, p),
                    c.name);
}

template <int MT, int NT, int EPI>
int launch_fp8(const Fp8Call& c, Fp8Params p, cudaStream_t st) {
  using S = Fp8Shape<MT, NT>;
  const void* kernel = reinterpret_cast<const void*>(fp8_gemm_kernel<MT, NT, EPI>);
  p.n_blocks = EPI == FP8_SWIGLU ? c.N / kWTile : (c.N + MT * kWTile - 1) / (MT * kWTile);
  long long units = 0;
  int rc = check_units(c, NT, p.n_blocks, &units);
  CUtensorMap tmW, tmA;
  if (rc == INVMOE_OK) rc = make_maps(c, p, NT, &tmW, &tmA);
  static std::atomic<uint64_t> attr_set{0};
  if (rc == INVMOE_OK) rc = set_smem_attr(kernel, S::SMEM_BYTES, attr_set);
  if constexpr (MT * NT >= 256) {
    static std::atomic<int> regs{0};
    if (rc == INVMOE_OK) rc = check_launch_regs(kernel, c.name, regs);
  }
  int sms = 0;
  if (rc == INVMOE_OK) rc = device_sm_count(&sms);
  if (rc) return rc;
  const unsigned grid = static_cast<unsigned>(units < sms ? units : sms);
  ProfScope prof(c.name, st);
  return check_cuda(launch_kernel(fp8_gemm_kernel<MT, NT, EPI>, dim3(grid), dim3(kFp8Threads), S::SMEM_BYTES, st, tmW,
                                  tmA, p),
                    c.name);
}

template <int MT, int EPI>
int launch_fp8_nt(const Fp8Call& c, const Fp8Params& p, long long per_group, cudaStream_t st) {
  if (per_group <= 16) return launch_fp8<MT, 16, EPI>(c, p, st);
  if (per_group <= 32) return launch_fp8<MT, 32, EPI>(c, p, st);
  if (per_group <= 64) return launch_fp8<MT, 64, EPI>(c, p, st);
  return launch_rows<EPI>(c, p, st);
}

}  // namespace

int fp8_gemm_run(const Fp8Call& c, cudaStream_t st) {
  if (c.rows == 0) return INVMOE_OK;
  Fp8Params p{};
  const bool swiglu = c.out_kind == FP8_OUT_SWIGLU;
  p.a_scale = c.a_scale;
  p.w_scale = c.w_scale;
  p.KB = (c.K + kFp8Block - 1) / kFp8Block;
  p.N = c.N;
  p.w_group_rows = swiglu ? 2 * c.N : c.N;
  p.w_srows = (p.w_group_rows + kFp8Block - 1) / kFp8Block;
  p.M = c.rows;
  p.G = c.G;
  p.counts = c.counts;
  p.offsets = c.offsets;
  p.out = c.out;
  p.out_scale = c.out_scale;
  p.vec_scale = p.KB % 4 == 0 && ((reinterpret_cast<uintptr_t>(c.a_scale) | reinterpret_cast<uintptr_t>(c.w_scale)) & 15) == 0;
  p.vec_out = c.N % 4 == 0;
  p.status = c.status;
  p.timeout_ns = kTimeoutNs;
  const long long per_group = c.G > 0 ? (static_cast<long long>(c.rows) + c.G - 1) / c.G : c.rows;
  if (swiglu) return launch_fp8_nt<2, FP8_SWIGLU>(c, p, per_group, st);
  if (c.out_kind == FP8_OUT_F32) return launch_fp8_nt<2, FP8_F32>(c, p, per_group, st);
  return launch_fp8_nt<2, FP8_BF16>(c, p, per_group, st);
}

}  // namespace invmoe
