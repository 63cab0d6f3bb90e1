// fp8_rows.cu -- the e4m3 product of many token rows (sm_103a; the arithmetic is described in fp8_gemm.cuh).
//
// Tokens are the MMA's M side: a CTA computes 128 token rows x 256 weight rows (one N = 256 MMA per K = 32
// step).  A thread holds one token row, so its scale is one number per block, read from global memory four blocks ahead:
// no shared memory on the scaling path, where the kernel of few tokens reads a scale for every column.
// Ten calls in a row on the same inputs: 8192 x 4096 x 6144 takes 166 us (2.48 PFLOP/s), 64 experts' gate and up of 2048 x
// 6144 with about 256 rows each 435 us; in a long run, under the power limit, the dense product takes 180.
// What bounds it is the handover of the products, 128 x 256 fp32 per block through two TMEM buffers: with the waits and
// arrives alone the dense product takes 134 us (a block is then 769 cycles: its 48 KB are written to shared memory and read
// from it, 768 cycles at 128 bytes; taking them from L2 at 64 bytes a cycle and SM would cost the same, and no measurement
// tells the two apart), with the loads from TMEM 147, with the 256 FFMA issue cycles per scheduler 169.  So a buffer is
// released as soon as its last columns are in registers, arrives are predicated, one elected thread issues, and how scales
// are loaded is known at compile time (169 -> 166).  Rows that do not start on 128 bytes (K % 128 != 0) cost a quarter more,
// since a box's rows then touch five sectors instead of four (4000 x 4096: K = 6144 95 us, 6160 121).
// Measured and not kept: CTA pairs with 256 x 256 tiles, 167 us, but 483 for those 64 experts, because the tiles are twice
// as high; loads of 16 columns, 175, or two loads of 32 at once, no change; blocks unrolled by two, 188; the last columns
// added behind the next block's wait, which spills, 229; packed fma.rn.f32x2, 690 instead of 485 cycles a block.
// SwiGLU: the 256 weight rows are 128 gate rows and the matching up rows.  A warpgroup has columns 64 half .. + 63 of
// either 128, so that a thread holds gate and up of the same h.
#include <type_traits>

#include "fp8_gemm.cuh"

namespace invmoe {

namespace {

// Registers per thread: 168 at launch (65,536 / 384, whole units of 8).  The tile leaves 128 accumulators in each of the
// 256 epilogue threads, so the first warpgroup hands registers over: 72 + 2 * 216 = 3 * 168.
constexpr int kLaunchRegs = 168, kLoaderRegs = 72, kEpiRegs = 216;
static_assert(kLoaderRegs + 2 * kEpiRegs <= 3 * kLaunchRegs, "register split");

// All four warps of a warpgroup execute the one instruction of its side of the split.
__device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoaderRegs)); }
__device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs)); }

struct Fp8RowsShape {
  static constexpr int TILE_BYTES = kWTile * kFp8Block;       // 16 KB: 128 rows x 128 e4m3
  static constexpr int STAGE_BYTES = 3 * TILE_BYTES;          // token rows, then two tiles of weight rows
  static constexpr int STAGES = 4;
  static constexpr int ACC_COLS = 256;
  static constexpr int ACC = 2;                               // TMEM buffers
  // output staging of a warp: 32 rows of 128 bytes for bulk stores, else 2 KB (store_rows)
  static constexpr int OSTAGE_BULK = kEpiWarps * 32 * 128;
  static constexpr int OSTAGE_PLAIN = kEpiWarps * 32 * 64;
  static constexpr int AMAX_BYTES = 2 * 2 * kWTile * 4;       // SwiGLU: [unit parity][warpgroup][row]
  static constexpr int BAR_BYTES = 256;
  static constexpr int smem_bytes(int groups, bool bulk, bool swiglu) {
    return 1024 + STAGES * STAGE_BYTES + (bulk ? OSTAGE_BULK : OSTAGE_PLAIN) + (swiglu ? AMAX_BYTES : 0) + BAR_BYTES +
           4 * (groups + 1) + 12;
  }
  static constexpr int SMEM_MAX = 232448;
  static_assert(8 * (2 * STAGES + 2 * ACC + 1) + 16 <= BAR_BYTES, "barriers");
};
static_assert(Fp8RowsShape::smem_bytes(kMaxGroups, false, true) <= Fp8RowsShape::SMEM_MAX &&
                  Fp8RowsShape::smem_bytes(256, true, false) <= Fp8RowsShape::SMEM_MAX,
              "shared memory");

// A warp's 32 rows x 16 * PIECES bytes from registers (one row per lane) to global memory, whole rows of 64 or 128 bytes
// at a time (PIECES lanes per row), through 2 KB of shared memory: 32 rows of 64 bytes, or twice 16 rows of 128.  The
// 16-byte piece c of row r sits at piece c ^ (r / 2 or r) of its row, free of bank conflicts both ways.
template <int ELT, int PIECES>
__device__ __forceinline__ void store_rows(uint8_t* stage, const uint32_t (&v)[4 * PIECES], uint8_t* out,
                                           long long ld_bytes, int rows_valid, long long bytes_valid, bool vec) {
  static_assert(PIECES == 4 || PIECES == 8, "64 or 128 bytes");
  constexpr int ROWS = 128 / PIECES;                   // rows staged at a time
  const int lane = threadIdx.x & 31;
  auto at = [&](int r, int c) { return stage + r * (16 * PIECES) + ((c ^ (PIECES == 8 ? r & 7 : (r >> 1) & 3)) << 4); };
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += ROWS) {
    if (lane >= r0 && lane < r0 + ROWS) {
#pragma unroll
      for (int k = 0; k < PIECES; ++k)
        *reinterpret_cast<uint4*>(at(lane - r0, k)) = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    }
    __syncwarp();
    if (vec) {
      const int c = lane % PIECES;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * (32 / PIECES) + lane / PIECES;
        const uint4 w = *reinterpret_cast<const uint4*>(at(r, c));
        if (r0 + r < rows_valid && c * 16 < bytes_valid) *reinterpret_cast<uint4*>(out + (r0 + r) * ld_bytes + c * 16) = w;
      }
    } else {
      // rows that start anywhere: one element per lane, so that a store still covers neighbouring bytes
      using E = std::conditional_t<ELT == 4, uint32_t, uint16_t>;
#pragma unroll 1
      for (int r = 0; r < ROWS && r0 + r < rows_valid; ++r) {
#pragma unroll
        for (int b = lane * ELT; b < 16 * PIECES; b += 32 * ELT)
          if (b < bytes_valid)
            *reinterpret_cast<E*>(out + (r0 + r) * ld_bytes + b) = *reinterpret_cast<const E*>(at(r, b >> 4) + (b & 15));
      }
    }
    __syncwarp();
  }
}

// VEC: scales in vectors of four blocks (p.vec_scale).
template <int EPI, bool VEC>
__global__ void __launch_bounds__(kFp8Threads, 1)
    fp8_rows_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
                    const __grid_constant__ CUtensorMap tmO, const Fp8Params p) {
  using S = Fp8RowsShape;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ostage = ring + S::STAGES * S::STAGE_BYTES;
  const bool bulk = EPI != FP8_SWIGLU && p.bulk_out != 0;
  float* s_amax = reinterpret_cast<float*>(ostage + (bulk ? S::OSTAGE_BULK : S::OSTAGE_PLAIN));
  uint64_t* full_bar =
      reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(s_amax) + (EPI == FP8_SWIGLU ? S::AMAX_BYTES : 0));
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
    if (warp == 0 && elect_one()) {
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
    } else if (warp == 1 && elect_one()) {
      // ---------------------------------------------------------- MMA issuer
      // To this thread all units are one stream of blocks.  It shares its scheduler with two epilogue warps, and what it
      // does between two blocks' MMAs the tensor cores wait for: the loop is unrolled over the ring, so that stages,
      // buffers, descriptors and barriers are constants (8192 x 4096 x 6144: a plain loop takes 5 us more).
      static_assert(S::STAGES == 4 && S::ACC == 2, "the unrolled stream");
      const uint64_t adesc0 = sdesc_k_sw128(smem_u32(ring));
      const uint64_t wdesc0 = sdesc_k_sw128(smem_u32(ring + S::TILE_BYTES));
      const uint32_t idesc = idesc_e4m3_f32(kWTile, S::ACC_COLS);
      const int my_units = total_units > static_cast<int>(blockIdx.x)
                               ? (total_units - 1 - static_cast<int>(blockIdx.x)) / static_cast<int>(gridDim.x) + 1
                               : 0;
      const long long blocks = static_cast<long long>(my_units) * p.KB;
      bool ok = true;
      uint32_t phase = 0;                              // of the ring; a buffer's second use in it has the other phase
      for (long long i0 = 0; ok && i0 < blocks; i0 += S::STAGES) {
#pragma unroll
        for (int s = 0; s < S::STAGES; ++s) {
          if (i0 + s >= blocks) break;
          const int acc = s & 1;
          const uint32_t acc_parity = s < 2 ? 1u : 0u;  // buffer `acc` for the (2 i / 4 + s / 2)-th time: even uses wait on 1
          if (!mbar_wait(&acce_bar[acc], acc_parity, wc) || !mbar_wait(&full_bar[s], phase, wc)) {
            ok = false;
            break;
          }
          tc_fence_after();
          uint64_t ad = adesc0, wd = wdesc0;
          asm volatile("" : "+l"(ad), "+l"(wd));       // descriptors of all stages at once would not fit the registers
          const uint64_t so = static_cast<uint64_t>((s * S::STAGE_BYTES) >> 4);
          const uint32_t d = tmem_base + static_cast<uint32_t>(acc * S::ACC_COLS);
#pragma unroll
          for (int kk = 0; kk < kFp8Block / 32; ++kk)
            umma_fp8(d, ad + so + 2u * kk, wd + so + 2u * kk, idesc, kk != 0 ? 1u : 0u);
          umma_commit(&accf_bar[acc]);
          umma_commit(&empty_bar[s]);
        }
        phase ^= 1u;
      }
      if (!ok) *s_abort = 1;
      // every MMA issued here has finished before the CTA releases TMEM
      umma_commit(final_bar);
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
    const int half = ew >> 2;                          // warpgroup: weight rows 64 half .. + 63 of either 128
    const int r_in_tile = q * 32 + lane;
    uint8_t* stg = ostage + ew * (bulk ? 32 * 128 : 32 * 64);
    const uint32_t on = lane == 0 ? 1u : 0u;
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
      float4 an = load_scales_as<VEC>(ap, 0, p), wn0 = load_scales_as<VEC>(wp0, 0, p), wn1 = load_scales_as<VEC>(wp1, 0, p);
      for (int kb0 = 0; kb0 < p.KB; kb0 += 4) {
        float4 ac = an, wc0 = wn0, wc1 = wn1;
        if (kb0 + 4 < p.KB) {
          an = load_scales_as<VEC>(ap, kb0 + 4, p);
          wn0 = load_scales_as<VEC>(wp0, kb0 + 4, p);
          wn1 = load_scales_as<VEC>(wp1, kb0 + 4, p);
        }
        const int n_kb = min(4, p.KB - kb0);
        // not unrolled (that measured slower): the scales of the next block move up instead
#pragma unroll 1
        for (int d = 0; d < n_kb; ++d) {
          const float s0 = __fmul_rn(ac.x, wc0.x), s1 = __fmul_rn(ac.x, wc1.x);
          ac.x = ac.y; ac.y = ac.z; ac.z = ac.w;
          wc0.x = wc0.y; wc0.y = wc0.z; wc0.z = wc0.w;
          wc1.x = wc1.y; wc1.y = wc1.z; wc1.z = wc1.w;
          if (ok && !mbar_test(&accf_bar[acc], acc_phase)) ok = mbar_wait_inline(&accf_bar[acc], acc_phase, wc);
          ok = __all_sync(0xffffffffu, ok);
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
                  // everything is in registers: the buffer is free before the last products are added.
                  // tcgen05.wait::ld has completed the warp's loads, so there is nothing left for a fence to order
                  mbar_arrive_if(on, &acce_bar[acc]);
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
          if (bulk) {
            // the previous piece has left the staging buffer
            if (lane == 0) bulk_wait_group_read0();
            __syncwarp();
          }
          if (bulk && rows_valid >= 32) {
            // a whole slab of the group: one bulk store of 32 rows x 128 bytes, clipped at N by the map, that drains
            // while this warp goes on
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<uint4*>(stg + lane * 128 + ((k ^ (lane & 7)) << 4)) =
                  make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&tmO, stg, n, static_cast<int>(row0));
              bulk_commit_group();
            }
          } else {
            store_rows<ELT, 8>(stg, w, static_cast<uint8_t*>(p.out) + row0 * ld + static_cast<long long>(n) * ELT, ld,
                               rows_valid, static_cast<long long>(p.N - n) * ELT, p.vec_out != 0);
          }
        }
      }
    }
    // the bulk stores this warp issued complete before the CTA exits
    if (bulk && lane == 0) bulk_wait_group0();
  }

  __syncwarp();                                       // the elected lanes rejoin their warps
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

template <int EPI, bool VEC>
int launch_rows(const Fp8Call& c, Fp8Params p, cudaStream_t st) {
  using S = Fp8RowsShape;
  const void* kernel = reinterpret_cast<const void*>(fp8_rows_kernel<EPI, VEC>);
  constexpr int ELT = EPI == FP8_F32 ? 4 : 2;
  constexpr bool SWIGLU = EPI == FP8_SWIGLU;
  p.n_blocks = SWIGLU ? c.N / kWTile : (c.N + 2 * kWTile - 1) / (2 * kWTile);
  p.vec_out = static_cast<long long>(c.N) * ELT % 16 == 0;
  // bulk stores where a tensor map can describe the output and its staging fits beside the groups' prefix sums
  p.bulk_out = !SWIGLU && p.vec_out && S::smem_bytes(c.G, true, false) <= S::SMEM_MAX;
  const int smem = S::smem_bytes(c.G, p.bulk_out != 0, SWIGLU);
  long long units = 0;
  int rc = check_units(c, kWTile, p.n_blocks, &units);
  CUtensorMap tmW, tmA, tmO{};
  if (rc == INVMOE_OK) rc = make_maps(c, p, kWTile, kWTile, 0, &tmW, &tmA);
  if (rc == INVMOE_OK && p.bulk_out) rc = make_tmap_out_rows(&tmO, c.out, ELT, c.N, c.rows);
  static std::atomic<uint64_t> attr_set{0};
  static std::atomic<int> regs{0};
  if (rc == INVMOE_OK) rc = set_smem_attr(kernel, S::SMEM_MAX, attr_set);
  if (rc == INVMOE_OK) rc = check_launch_regs(kernel, c.name, regs);
  int sms = 0;
  if (rc == INVMOE_OK) rc = device_sm_count(&sms);
  if (rc) return rc;
  const unsigned grid = static_cast<unsigned>(units < sms ? units : sms);
  ProfScope prof(c.name, st);
  return check_cuda(launch_kernel(fp8_rows_kernel<EPI, VEC>, dim3(grid), dim3(kFp8Threads), static_cast<size_t>(smem), st, tmW,
                                  tmA, tmO, p),
                    c.name);
}

}  // namespace

int fp8_rows_run(const Fp8Call& c, const Fp8Params& p, cudaStream_t st) {
  if (c.out_kind == FP8_OUT_SWIGLU) return p.vec_scale ? launch_rows<FP8_SWIGLU, true>(c, p, st) : launch_rows<FP8_SWIGLU, false>(c, p, st);
  if (c.out_kind == FP8_OUT_F32) return p.vec_scale ? launch_rows<FP8_F32, true>(c, p, st) : launch_rows<FP8_F32, false>(c, p, st);
  return p.vec_scale ? launch_rows<FP8_BF16, true>(c, p, st) : launch_rows<FP8_BF16, false>(c, p, st);
}

}  // namespace invmoe
