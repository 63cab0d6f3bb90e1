// fp8_cols.cu -- the e4m3 product of few token rows per weight (sm_103a; the arithmetic is described in fp8_gemm.cuh).
//
// Weights are the MMA's M side (MT sub-tiles of WR rows; a sub-tile lies in one scale block, so its scale is one number
// per block of K) and tokens its N side, in multiples of 16: a group of 20 tokens costs 32 columns, not 128 rows.
// What bounds it is reading the weights (4 tokens that reach 24 of 64 experts of 2 x 2048 x 6144, 604 MB: 95 us, 6.3 TB/s of
// DRAM), and, for one small matrix, latency: a step of KS K blocks goes through every handover at once (one copy per operand,
// one ring stage, one TMEM buffer, one set of scales, one wait of each role), and where 256-row tiles would leave SMs without
// work 64-row tiles are used (8 x 4096 x 6144: 64 CTAs instead of 16; 8 us, of which 2 until the first block is there, 4 for
// twelve steps and the rest launch and output; 32-row tiles on 128 CTAs: 8.5).
//   * warp 0: one thread copies; with K % 128 == 0 the KS blocks of a box come in one rank-3 copy;
//   * warp 1: one thread issues the MMAs, 4 K = 32 steps per block and sub-tile, each block into columns of its own;
//   * warps 2 and 3: the scales, from global memory four blocks ahead, into the slot of the TMEM buffer they belong to
//     (its barrier counts the MMAs' commit and these two warps);
//   * two warpgroups, each with half of the token columns and all lanes.  TMEM is read in the 16x256b shape: a thread
//     then holds 2 or 4 rows x NT/8 columns instead of one row x NT/2, so it needs a quarter of the tokens' scales.
// SwiGLU (MT = 2, WR = 128): sub-tile 0 holds 128 gate rows, sub-tile 1 the matching up rows; h = silu(g) * u, its absolute
// maximum over the 128 rows, and e4m3(h / scale) leave the kernel, never g, u or an unquantised h.
#include "fp8_gemm.cuh"

namespace invmoe {

namespace {

constexpr int kScaleWarps = 2;
constexpr int kStageF32 = kWTile + 4;               // floats per staged token row (conflict-free fragment writes)
constexpr int kStageFp8 = kWTile + 16;              // bytes per staged token row
constexpr int kStagingBytes = 8448;                 // per warpgroup: 16 x 132 floats or 32 x 144 bytes
static_assert(16 * kStageF32 * 4 <= kStagingBytes && 32 * kStageFp8 <= kStagingBytes, "staging");

template <int MT, int WR, int NT, int KS>
struct Fp8ColsShape {
  static constexpr int W_BYTES = WR * kFp8Block;                        // one block of one sub-tile
  static constexpr int A_BYTES = NT * kFp8Block;
  static constexpr int STAGE_BYTES = KS * (MT * W_BYTES + A_BYTES);     // [sub-tile][block][row], then [block][token]
  static constexpr int STEP_COLS = KS * MT * NT;
  static constexpr int ACC = 512 / STEP_COLS < 4 ? 512 / STEP_COLS : 4; // TMEM buffers
  static constexpr int TMEM_COLS = ACC * STEP_COLS < 32 ? 32 : ACC * STEP_COLS;
  static constexpr int HALF = NT / 2;                                   // token columns of a warpgroup
  static constexpr int BLOCK_SCALES = NT + 4;                           // NT tokens, MT weight blocks
  static constexpr int SCALE_BYTES = ACC * KS * BLOCK_SCALES * 4;
  static constexpr int AMAX_BYTES = 2 * 4 * HALF * 4;                   // [warpgroup][warp][column]
  static constexpr int BAR_BYTES = 256;
  static constexpr int FIXED = 1024 + 2 * kStagingBytes + SCALE_BYTES + AMAX_BYTES + BAR_BYTES + 4 * (kMaxGroups + 1) + 12;
  static constexpr int STAGES = (232448 - FIXED) / STAGE_BYTES < 8 ? (232448 - FIXED) / STAGE_BYTES : 8;
  static constexpr int SMEM_BYTES = FIXED + STAGES * STAGE_BYTES;
  static_assert(SMEM_BYTES <= 232448 && STAGES >= 3, "shared memory");
  static_assert(STAGE_BYTES % 1024 == 0, "swizzle atoms");
  static_assert(8 * (2 * STAGES + 2 * ACC + 1) + 16 <= BAR_BYTES, "barriers");
};

// 16 TMEM lanes x 8 * X columns (16x256b shape): register 4i + {0, 1} holds lane t / 4, columns 8i + 2(t % 4) + {0, 1},
// register 4i + {2, 3} the same columns of lane t / 4 + 8 (t = lane of the warp).
template <int X>
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t taddr, uint32_t (&r)[4 * X]) {
  static_assert(X == 1 || X == 2 || X == 4, "repeat");
  if constexpr (X == 1) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
  } else if constexpr (X == 2) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  }
}

// The registers are seen as redefined here (after tcgen05.wait::ld), so no use of them moves above the wait.
template <int R>
__device__ __forceinline__ void reg_fence(uint32_t (&r)[R]) {
#pragma unroll
  for (int i = 0; i < R; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ void bar_wg(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

template <int MT, int WR, int NT, int KS, int EPI>
__global__ void __launch_bounds__(kFp8Threads, 1)
    fp8_cols_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
                    const Fp8Params p) {
  using S = Fp8ColsShape<MT, WR, NT, KS>;
  static_assert(EPI != FP8_SWIGLU || (MT == 2 && WR == kWTile), "SwiGLU pairs a gate sub-tile with its up sub-tile");
  static_assert(WR == 64 || WR == 128, "MMA rows");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = ring + S::STAGES * S::STAGE_BYTES;
  float* s_scale = reinterpret_cast<float*>(staging + 2 * kStagingBytes);
  float* s_amax = s_scale + S::SCALE_BYTES / 4;
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
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int a = 0; a < S::ACC; ++a) {
      mbar_init(&accf_bar[a], 1 + kScaleWarps);
      mbar_init(&acce_bar[a], kEpiWarps);
    }
    mbar_init(final_bar, 1);
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
  const int steps = (p.KB + KS - 1) / KS;
  WaitCtl wc{s_abort, p.status, p.timeout_ns};

  if (warp == 0) {
    if (elect_one()) {
      // ---------------------------------------------------------- producer
      int stage = 0;
      uint32_t phase = 0;
      int fills = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < total_units; u += gridDim.x) {
        const Fp8Unit U = fp8_unit<NT>(u, p, s_prefix, total_chunks);
        const int w_row = U.g * p.w_group_rows + (EPI == FP8_SWIGLU ? U.nb * WR : U.nb * MT * WR);
        const int w_next = EPI == FP8_SWIGLU ? p.N : WR;             // from one sub-tile's rows to the next one's
        for (int st = 0; st < steps; ++st) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1u, wc)) { ok = false; break; }
          uint8_t* sw = ring + stage * S::STAGE_BYTES;
          uint8_t* sa = sw + KS * MT * S::W_BYTES;
          // a box counts its full size, rows and blocks filled with zeros included
          if (KS > 1 && p.k_boxes) {
            mbar_arrive_expect_tx(&full_bar[stage], S::STAGE_BYTES);
#pragma unroll
            for (int m = 0; m < MT; ++m)
              tma_load_3d(sw + m * KS * S::W_BYTES, &tmW, &full_bar[stage], 0, w_row + m * w_next, st * KS);
            tma_load_3d(sa, &tmA, &full_bar[stage], 0, U.row0, st * KS);
          } else {
            const int n = min(KS, p.KB - st * KS);
            mbar_arrive_expect_tx(&full_bar[stage], static_cast<uint32_t>(n * (S::STAGE_BYTES / KS)));
            for (int ks = 0; ks < n; ++ks) {
              const int c = (st * KS + ks) * kFp8Block;
#pragma unroll
              for (int m = 0; m < MT; ++m)
                tma_load_2d(sw + (m * KS + ks) * S::W_BYTES, &tmW, &full_bar[stage], c, w_row + m * w_next);
              tma_load_2d(sa + ks * S::A_BYTES, &tmA, &full_bar[stage], c, U.row0);
            }
          }
          ++fills;
          if (++stage == S::STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // every copy this thread issued lands before the CTA can exit
      WaitCtl drain{nullptr, p.status, p.timeout_ns};
      for (int s = 0; s < S::STAGES && s < fills; ++s)   // the last of this stage's fills
        mbar_wait(&full_bar[s], static_cast<uint32_t>((fills - 1 - s) / S::STAGES) & 1u, drain);
    }
  } else if (warp == 1) {
    if (elect_one()) {
      // ---------------------------------------------------------- MMA issuer
      const uint64_t wdesc0 = sdesc_k_sw128(smem_u32(ring));
      const uint64_t adesc0 = sdesc_k_sw128(smem_u32(ring + KS * MT * S::W_BYTES));
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < total_units; u += gridDim.x) {
        const Fp8Unit U = fp8_unit<NT>(u, p, s_prefix, total_chunks);
        const uint32_t idesc = idesc_e4m3_f32(WR, (U.cols + 15) & ~15);
        for (int st = 0; st < steps; ++st) {
          if (!mbar_wait(&acce_bar[acc], acc_phase ^ 1u, wc) || !mbar_wait(&full_bar[stage], phase, wc)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t so = static_cast<uint64_t>((stage * S::STAGE_BYTES) >> 4);
          const uint32_t d0 = tmem_base + static_cast<uint32_t>(acc * S::STEP_COLS);
          const int n = min(KS, p.KB - st * KS);
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            if (ks < n) {
#pragma unroll
              for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int kk = 0; kk < kFp8Block / 32; ++kk)   // K = 32 steps: 32 bytes on inside the swizzle row
                  umma_fp8(d0 + static_cast<uint32_t>((ks * MT + m) * NT),
                           wdesc0 + so + static_cast<uint64_t>((m * KS + ks) * (S::W_BYTES >> 4)) + 2u * kk,
                           adesc0 + so + static_cast<uint64_t>(ks * (S::A_BYTES >> 4)) + 2u * kk, idesc,
                           kk != 0 ? 1u : 0u);
            }
          }
          umma_commit(&accf_bar[acc]);
          umma_commit(&empty_bar[stage]);
          if (++stage == S::STAGES) { stage = 0; phase ^= 1u; }
          if (++acc == S::ACC) { acc = 0; acc_phase ^= 1u; }
        }
      }
      if (!ok) *s_abort = 1;
      // every MMA issued here has finished before the CTA releases TMEM
      umma_commit(final_bar);
      WaitCtl drain{nullptr, p.status, p.timeout_ns};
      mbar_wait(final_bar, 0, drain);
    }
  } else if (warp < kFirstEpiWarp) {
    // ------------------------------------------------------------ scales: thread j has token j's, threads below MT the
    // weight blocks' as well
    const int j = (warp - 2) * 32 + lane;
    const bool on_a = j < NT, on_w = j < MT;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < total_units; u += gridDim.x) {
      const Fp8Unit U = fp8_unit<NT>(u, p, s_prefix, total_chunks);
      const float* ap = p.a_scale + static_cast<long long>(U.row0 + min(j, U.cols - 1)) * p.KB;
      const int srow = EPI == FP8_SWIGLU ? U.nb + j * (p.N / kFp8Block) : (U.nb * MT + j) * WR / kWTile;
      const float* wp = p.w_scale + (static_cast<long long>(U.g) * p.w_srows + min(srow, p.w_srows - 1)) * p.KB;
      float4 an = make_float4(0.f, 0.f, 0.f, 0.f), wn = an;
      if (on_a) an = load_scales(ap, 0, p);
      if (on_w) wn = load_scales(wp, 0, p);
      for (int kb0 = 0; ok && kb0 < p.KB; kb0 += 4) {
        const float av[4] = {an.x, an.y, an.z, an.w}, wv[4] = {wn.x, wn.y, wn.z, wn.w};
        if (kb0 + 4 < p.KB) {
          if (on_a) an = load_scales(ap, kb0 + 4, p);
          if (on_w) wn = load_scales(wp, kb0 + 4, p);
        }
#pragma unroll
        for (int d = 0; d < 4; d += KS) {
          if (kb0 + d >= p.KB) break;
          ok = wait_warp(&acce_bar[acc], acc_phase ^ 1u, wc);
          if (!ok) break;
          float* slot = s_scale + acc * (KS * S::BLOCK_SCALES);
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            if (on_a) slot[ks * S::BLOCK_SCALES + j] = av[d + ks];
            if (on_w) slot[ks * S::BLOCK_SCALES + NT + j] = wv[d + ks];
          }
          __syncwarp();
          mbar_arrive_if(lane == 0 ? 1u : 0u, &accf_bar[acc]);
          if (++acc == S::ACC) { acc = 0; acc_phase ^= 1u; }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ scaling and epilogue
    // All eight warps walk the same units whatever happens, so the warpgroup barriers always meet; after a wait that ran
    // out (ok = false) a warp only keeps those barriers.
    constexpr int X = NT / 16;                         // 8-column fragments of a warpgroup's columns
    constexpr int HL = WR / 64;                        // 16-lane halves in use (M = 64 fills lanes 0..15 of a quadrant)
    const int q = warp & 3;                            // TMEM lane quadrant
    const int half = (warp - kFirstEpiWarp) >> 2;      // warpgroup: token columns [half * HALF, +HALF)
    const int tid = q * 32 + lane;                     // thread of the warpgroup
    const int bar_id = 1 + half;
    const uint32_t on = lane == 0 ? 1u : 0u;
    float* my_amax = s_amax + half * (4 * S::HALF);
    uint8_t* stg = staging + half * kStagingBytes;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < total_units; u += gridDim.x) {
      const Fp8Unit U = fp8_unit<NT>(u, p, s_prefix, total_chunks);
      const int wg_cols = U.cols - half * S::HALF;     // this warpgroup's tokens (may be <= 0)
      float v[MT][HL][4 * X];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < HL; ++h)
#pragma unroll
          for (int i = 0; i < 4 * X; ++i) v[m][h][i] = 0.0f;
      for (int st = 0; st < steps; ++st) {
        if (ok) ok = wait_warp(&accf_bar[acc], acc_phase, wc);
        if (ok) {
          const int n = min(KS, p.KB - st * KS);
          uint32_t r[KS][MT][HL][4 * X];
          float2 sa[KS][X];
          float sw[KS][MT];
          if (wg_cols > 0) {
            tc_fence_after();
            const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                static_cast<uint32_t>(acc * S::STEP_COLS + half * S::HALF);
            // blocks past the last are read too (whatever the columns hold) and not used
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
              for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < HL; ++h)
                  tmem_ld_16x256b<X>(tb + (static_cast<uint32_t>(h * 16) << 16) + static_cast<uint32_t>((ks * MT + m) * NT),
                                     r[ks][m][h]);
            const float* slot = s_scale + acc * (KS * S::BLOCK_SCALES);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
              for (int i = 0; i < X; ++i)
                sa[ks][i] = *reinterpret_cast<const float2*>(slot + ks * S::BLOCK_SCALES + half * S::HALF + 8 * i +
                                                             2 * (lane & 3));
#pragma unroll
              for (int m = 0; m < MT; ++m) sw[ks][m] = slot[ks * S::BLOCK_SCALES + NT + m];
            }
            tmem_ld_wait();
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
              for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < HL; ++h) reg_fence(r[ks][m][h]);
            tc_fence_before();
          }
          // products and scales are in registers: the buffer and its slot are free
          __syncwarp();
          mbar_arrive_if(on, &acce_bar[acc]);
          if (wg_cols > 0) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
              if (ks < n) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                  for (int i = 0; i < X; ++i) {
                    const float s0 = __fmul_rn(sa[ks][i].x, sw[ks][m]), s1 = __fmul_rn(sa[ks][i].y, sw[ks][m]);
#pragma unroll
                    for (int h = 0; h < HL; ++h)
#pragma unroll
                      for (int e = 0; e < 4; ++e)
                        v[m][h][4 * i + e] = fmaf(__uint_as_float(r[ks][m][h][4 * i + e]), e & 1 ? s1 : s0, v[m][h][4 * i + e]);
                  }
              }
            }
          }
        }
        if (++acc == S::ACC) { acc = 0; acc_phase ^= 1u; }
      }
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
            for (int h = 0; h < HL; ++h)
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
        if (tid < S::HALF)
          my_s = fp8_scale(fmaxf(fmaxf(my_amax[tid], my_amax[S::HALF + tid]),
                                 fmaxf(my_amax[2 * S::HALF + tid], my_amax[3 * S::HALF + tid])));
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
            for (int h = 0; h < HL; ++h)
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
          const int n0 = (U.nb * MT + m) * WR;
#pragma unroll
          for (int i0 = 0; i0 < X; i0 += CI) {
            bar_wg(bar_id);
#pragma unroll
            for (int ii = 0; ii < CI; ++ii)
#pragma unroll
              for (int h = 0; h < HL; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  stf[(8 * ii + 2 * (lane & 3) + (e & 1)) * kStageF32 + q * (WR / 4) + 16 * h + 8 * (e >> 1) + (lane >> 2)] =
                      v[m][h][4 * (i0 + ii) + e];
            bar_wg(bar_id);
            // one warp per token row: 4 outputs per lane
#pragma unroll
            for (int tt = q; tt < 8 * CI; tt += 4) {
              const int t = 8 * i0 + tt;
              const int n = n0 + 4 * lane;
              if (!ok || t >= wg_cols || 4 * lane >= WR || n >= p.N) continue;
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

  __syncwarp();                                       // the elected lanes rejoin their warps
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, S::TMEM_COLS);
  }
}

template <int MT, int WR, int NT, int KS, int EPI>
int launch_cols(const Fp8Call& c, Fp8Params p, cudaStream_t st) {
  using S = Fp8ColsShape<MT, WR, NT, KS>;
  p.n_blocks = EPI == FP8_SWIGLU ? c.N / WR : (c.N + MT * WR - 1) / (MT * WR);
  p.vec_out = c.N % 4 == 0;
  p.k_boxes = KS > 1 && c.K % kFp8Block == 0;
  long long units = 0;
  int rc = check_units(c, NT, p.n_blocks, &units);
  CUtensorMap tmW, tmA;
  if (rc == INVMOE_OK) rc = make_maps(c, p, WR, NT, p.k_boxes ? KS : 0, &tmW, &tmA);
  static std::atomic<uint64_t> attr_set{0};
  if (rc == INVMOE_OK)
    rc = set_smem_attr(reinterpret_cast<const void*>(fp8_cols_kernel<MT, WR, NT, KS, EPI>), S::SMEM_BYTES, attr_set);
  int sms = 0;
  if (rc == INVMOE_OK) rc = device_sm_count(&sms);
  if (rc) return rc;
  const unsigned grid = static_cast<unsigned>(units < sms ? units : sms);
  ProfScope prof(c.name, st);
  return check_cuda(launch_kernel(fp8_cols_kernel<MT, WR, NT, KS, EPI>, dim3(grid), dim3(kFp8Threads), S::SMEM_BYTES,
                                  st, tmW, tmA, p),
                    c.name);
}

template <int EPI>
int launch_plain(const Fp8Call& c, const Fp8Params& p, int nt, bool small, cudaStream_t st) {
  if (nt == 64) return launch_cols<1, 64, 64, 2, EPI>(c, p, st);
  if (small)
    return nt == 16 ? launch_cols<1, 64, 16, 4, EPI>(c, p, st) : launch_cols<1, 64, 32, 4, EPI>(c, p, st);
  return nt == 16 ? launch_cols<2, 128, 16, 2, EPI>(c, p, st) : launch_cols<2, 128, 32, 1, EPI>(c, p, st);
}

}  // namespace

// Which kernel and tile: by the rows of a group (all rows of a dense call; the average, half as much again for the spread
// around it, of a grouped one) and by what fills the machine.
//   * at most 64 rows: columns, in 16, 32 or 64.  With 16 or 32 the tile is 256 weight rows (4 tokens that reach 24 of
//     64 experts of 6144 x 2048, 302 MB: 49.7 us, with 64-row tiles 51.5), or 64 where that would not give every SM one (8 x 4096 x 6144: 8 us); with
//     64, where a step holds fewer blocks of the larger tile, 64 rows (256 tokens, all 64 experts: 143 us against 156);
//   * more: the row tiles (512 tokens, the same experts: 154 us against 210 in columns), unless the 64-row tiles are done
//     in two waves, when 128-row tiles leave most SMs idle (128 x 4096 x 6144: 12 us against 26, 256 rows: 20 against 26,
//     320 rows, three waves: 28 against 26).
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
  p.vec_scale = p.KB % 4 == 0 &&
                ((reinterpret_cast<uintptr_t>(c.a_scale) | reinterpret_cast<uintptr_t>(c.w_scale)) & 15) == 0;
  p.status = c.status;
  p.timeout_ns = kTimeoutNs;
  long long rows = c.rows;
  if (c.G > 0) {
    rows = (rows + c.G - 1) / c.G;
    rows += rows / 2;
  }
  const int nt = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  if (swiglu) {
    if (rows > 64) return fp8_rows_run(c, p, st);
    if (nt == 16) return launch_cols<2, 128, 16, 2, FP8_SWIGLU>(c, p, st);
    if (nt == 32) return launch_cols<2, 128, 32, 1, FP8_SWIGLU>(c, p, st);
    return launch_cols<2, 128, 64, 1, FP8_SWIGLU>(c, p, st);
  }
  long long units256 = 0, units64 = 0;
  int sms = 0;
  int rc = check_units(c, nt, (c.N + 2 * kWTile - 1) / (2 * kWTile), &units256);
  if (rc == INVMOE_OK) rc = check_units(c, nt, (c.N + 63) / 64, &units64);
  if (rc == INVMOE_OK) rc = device_sm_count(&sms);
  if (rc) return rc;
  if (rows > 64 && units64 > 2 * sms) return fp8_rows_run(c, p, st);
  const bool small = units256 < sms;
  return c.out_kind == FP8_OUT_F32 ? launch_plain<FP8_F32>(c, p, nt, small, st)
                                   : launch_plain<FP8_BF16>(c, p, nt, small, st);
}

}  // namespace invmoe
