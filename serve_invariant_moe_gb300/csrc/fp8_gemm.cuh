// fp8_gemm.cuh -- what the two e4m3 product kernels (fp8_cols.cu, fp8_rows.cu) share (sm_103a).
//
//   out[t, n] = sum_kb (as[t, kb] * ws[n / 128, kb]) * p_kb[t, n],   p_kb = sum_{k in block kb} a[t, k] * w[n, k]
//
// p_kb comes from the tensor cores (tcgen05 kind::f8f6f4, four K = 32 steps, fp32 in TMEM, a fresh accumulator for every
// block); its scale is an arbitrary fp32 number, so the sum over blocks cannot stay in TMEM: epilogue warps read each
// p_kb and keep acc = fma(p_kb, as * ws, acc) in fp32 registers, kb ascending.  No split of K, one order in both kernels
// and every tile shape, and a token's chain depends on that token only: the bits do not depend on the batch.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "fp8.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace invmoe {

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
  int vec_out;              // output rows are a multiple of the store vector
  int k_boxes;              // several blocks per copy (rank-3 tensor maps)
  int bulk_out;             // whole 32-row slabs leave by bulk tensor stores
  unsigned int* status;
  unsigned long long timeout_ns;
};

constexpr int kWTile = 128;                         // weight rows that share a scale
constexpr int kMaxGroups = 1024;
constexpr int kEpiWarps = 8;
constexpr int kFirstEpiWarp = 4;                    // warps 0..3: producer, MMA issuer, and what each kernel says
constexpr int kFp8Threads = 32 * (kFirstEpiWarp + kEpiWarps);

// Instruction descriptor, kind::f8f6f4: e4m3 A and B (formats 0), fp32 D, both K-major.
__device__ __forceinline__ uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// One lane of a converged warp, the same one every time.  What issues copies and MMAs runs under it: these instructions take
// their operands from uniform registers, and only where the compiler knows that one thread executes does it keep
// descriptors there.  Under a test of the lane number each MMA cost 60 to 100 cycles, predicated or branched around;
// elected 20 (8 x 4096 x 6144: 13.4 -> 8.0 us).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r));
  return r != 0;
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

// Arrive of the lane whose `on` is set.  Predicated: a branch of one lane, its reconvergence included, cost an epilogue warp
// some 120 of 1040 cycles a block (8192 x 4096 x 6144: 187 -> 170 us).
__device__ __forceinline__ void mbar_arrive_if(uint32_t on, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(on)
      : "memory");
}

// silu(g) * u = g / (1 + exp(-g)) * u in fp32: expf's error does not grow with |g|, as the hardware's exponential's does, and
// h's fp32 scale would show it.  The quotient is a product with a reciprocal that is within one unit in the last place: an
// exact division costs the gate/up product 20 % more (8192 tokens, 256 experts of 2 x 2048 x 6144: 2130 us against 1730;
// with __expf the same as this to 3 %).  A quarter of the denominator keeps the reciprocal a normal number up to the largest
// exp(-g); above it, it is 0, as the quotient is.  Both kernels use this expression, so h does not depend on which one runs.
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float swiglu(float g, float u) {
  return __fmul_rn(__fmul_rn(0.25f * g, rcp_approx(fmaf(expf(-g), 0.25f, 0.25f))), u);
}

// mbar_wait by a whole warp, one answer for all lanes.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, const WaitCtl& w) {
  if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait_slow(bar, parity, w));
}

// Scales of blocks kb .. kb + 3 of one row (past the last: the last one's, which nothing uses); VEC: p.vec_scale.
template <bool VEC>
__device__ __forceinline__ float4 load_scales_as(const float* src, int kb, const Fp8Params& p) {
  if (VEC) return __ldg(reinterpret_cast<const float4*>(src + kb));
  const int last = p.KB - 1;
  return make_float4(__ldg(src + kb), __ldg(src + min(kb + 1, last)), __ldg(src + min(kb + 2, last)),
                     __ldg(src + min(kb + 3, last)));
}

// Which of the two at run time, for a kernel that loads few.
__device__ __forceinline__ float4 load_scales(const float* src, int kb, const Fp8Params& p) {
  return p.vec_scale ? load_scales_as<true>(src, kb, p) : load_scales_as<false>(src, kb, p);
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
    if (lane == 0) *total = (p.M - 1) / CH + 1;
    return;
  }
  auto chunks = [](int n) { return n / CH + (n % CH != 0); };
  const int per = (p.G + 31) / 32;
  const int g0 = lane * per;
  int local = 0;
  for (int i = 0; i < per; ++i)
    if (g0 + i < p.G) local += chunks(__ldg(p.counts + g0 + i));
  int incl = local;
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  int run = incl - local;
  for (int i = 0; i < per; ++i)
    if (g0 + i < p.G) {
      prefix[g0 + i] = run;
      run += chunks(__ldg(p.counts + g0 + i));
    }
  if (lane == 31) {
    prefix[p.G] = incl;
    *total = incl;
  }
}

// Host side: the largest number of units of a call, and the tensor maps.
inline int check_units(const Fp8Call& c, int chunk, int n_blocks, long long* units) {
  const long long chunks = c.G > 0 ? static_cast<long long>(c.rows) / chunk + (c.rows < c.G ? c.rows : c.G)
                                   : (static_cast<long long>(c.rows) + chunk - 1) / chunk;
  *units = chunks * n_blocks;
  // below 2^31 by more than a grid, so that a CTA's unit index cannot pass it either
  if (*units > 0x7fff0000LL) return set_error(INVMOE_ERR_UNSUPPORTED_SHAPE, "%s: too many tiles for one launch", c.name);
  return INVMOE_OK;
}

// Weights in boxes of w_box rows, tokens in boxes of a_box rows; k_blocks > 0: rank-3 boxes of that many blocks along K.
inline int make_maps(const Fp8Call& c, const Fp8Params& p, int w_box, int a_box, int k_blocks, CUtensorMap* w,
                     CUtensorMap* a) {
  const int rc = make_tmap_fp8(w, c.w, c.K, static_cast<long long>(p.w_group_rows) * (c.G > 0 ? c.G : 1), w_box, k_blocks);
  return rc ? rc : make_tmap_fp8(a, c.a, c.K, c.rows, a_box, k_blocks);
}

int fp8_rows_run(const Fp8Call& c, const Fp8Params& p, cudaStream_t st);

}  // namespace invmoe
