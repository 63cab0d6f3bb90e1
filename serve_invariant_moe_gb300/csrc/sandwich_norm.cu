// sandwich_norm.cu -- the norms after and before a block in one pass, and their backward.
//
//   n = x rstd_p w_p,  r' = a r + b g n  (stored in the residual's type),  y = r' rstd w_n
//
// with rstd_p = 1 / sqrt(mean(x^2) + eps) of the block's output x, rstd likewise of the stored row r', a and b scalars and
// the gate g one number per channel or per token (or absent).  Bound by memory: per element the forward reads x and r and
// writes r' and y.  One block holds one row in registers across both sums; the reduction orders depend on H alone.
// 8192 x 6144, fp32 x, bf16 residual, a channel's gate: 78.3 us for 503 MB, 6.4 TB/s (82.5 with 51 registers, where 40 leave
// room for another block, 80.0 with the warps' sums read one by one); 8 rows: 7 us, the host's call.  The 40 registers spill 8
// bytes there, 44 to 60 with an fp32 residual (116 us, 6.1 TB/s); the 64 above 8192 columns 12 to 132 (2048 x 16384: 5.5 TB/s
// with a bf16 residual, 4.4 with fp32).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"
#include "row_ops.cuh"

namespace invmoe {

namespace {

struct Gate {
  const __nv_bfloat16* channel;   // [H] or null
  const float* token;             // [T] or null
};

// What multiplies the normalised row apart from its weight: b times the gate of 8 channels or of the row.
__device__ __forceinline__ void branch_factor(const Gate& gate, float branch_scale, float token, int c, float (&f)[8]) {
  if (gate.channel != nullptr) {
    load8(gate.channel + c, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(f[i], branch_scale);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = token;
  }
}

__device__ __forceinline__ float token_factor(const Gate& gate, float branch_scale, long long t) {
  return gate.token != nullptr ? __fmul_rn(__ldg(gate.token + t), branch_scale) : branch_scale;
}

__device__ __forceinline__ float inv_rms(float ss, int H, float eps) {
  return __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(ss, static_cast<float>(H)), eps)));
}

// block_sum with the same order of additions, four of the warps' sums to a load.
__device__ __forceinline__ float block_sum4(float v, float* s_part, int warp, int lane, int nwarps) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  if (nwarps == 1) return v;
  if (lane == 0) s_part[warp] = v;
  __syncthreads();
  float s = 0.0f;
  int w = 0;
  for (; w + 4 <= nwarps; w += 4) {
    const float4 t = *reinterpret_cast<const float4*>(s_part + w);
    s += t.x;
    s += t.y;
    s += t.z;
    s += t.w;
  }
  for (; w < nwarps; ++w) s += s_part[w];
  return s;
}

template <int V, typename TX, typename TR>
__global__ void __launch_bounds__(max_threads(V), V == 2 ? 3 : 1)
    sandwich_kernel(const TX* __restrict__ x, const __nv_bfloat16* __restrict__ w_post, const TR* res, const Gate gate,
                    const __nv_bfloat16* __restrict__ w_next, int H, float res_scale, float branch_scale, float eps,
                    TR* res_out, __nv_bfloat16* __restrict__ out, uint8_t* __restrict__ q, float* __restrict__ scale,
                    float* __restrict__ rstd_post, float* __restrict__ rstd_out) {
  pdl_wait();
  pdl_trigger();
  __shared__ __align__(16) float s_part[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
  const long long t = blockIdx.x;
  const long long base = t * H;
  float r[V][8];
  Raw8<TR> old[V];
  float ss = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * blockDim.x + threadIdx.x) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[v][i] = 0.0f;
    old[v].zero();
    if (c < H) {
      load8(x + base + c, r[v]);
      old[v].load(res + base + c);
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(r[v][i], r[v][i], ss);
  const float rstd_p = inv_rms(block_sum4(ss, s_part[0], warp, lane, nwarps), H, eps);
  const float token = token_factor(gate, branch_scale, t);
  ss = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * blockDim.x + threadIdx.x) * 8;
    if (c < H) {
      float w[8], f[8], b[8];
      load8(w_post + c, w);
      branch_factor(gate, branch_scale, token, c, f);
      old[v].get(b);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        r[v][i] = __fadd_rn(__fmul_rn(b[i], res_scale), __fmul_rn(__fmul_rn(__fmul_rn(r[v][i], rstd_p), w[i]), f[i]));
      // the second norm reads the row as it is stored: the next layer and the backward see the same one
      store8(res_out + base + c, r[v]);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(r[v][i], r[v][i], ss);
    }
  }
  if (rstd_post != nullptr && threadIdx.x == 0) rstd_post[t] = rstd_p;
  if (w_next == nullptr) return;
  const float rstd = inv_rms(block_sum4(ss, s_part[1], warp, lane, nwarps), H, eps);
  if (rstd_out != nullptr && threadIdx.x == 0) rstd_out[t] = rstd;
  const int nb = (H + kFp8Block - 1) / kFp8Block;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * blockDim.x + threadIdx.x) * 8;
    const bool in = c < H;
    float w[8], y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0.0f;
    if (in) load8(w_next + c, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = in ? __fmul_rn(__fmul_rn(r[v][i], rstd), w[i]) : 0.0f;
    if (q != nullptr) quant8(y, in, q + base + c, scale + t * nb + c / kFp8Block, lane);
    if (out != nullptr && in) store8(out + base + c, y);
  }
}

// Backward.  With r^ = r' rstd and n^ = x rstd_p, rounding passed straight through:
//   e = dy w_n,  d = dres + rstd (e - r^ mean(e r^))               the gradient of r'
//   dresidual = a d,  u = b g d w_p,  dx = rstd_p (u - n^ mean(u n^))
//   dw_n = sum_t dy r^,  dw_p = b sum_t g d n^,  dg = b sum_t d w_p n^ (a channel's) or b sum_h d w_p n^ (a token's)
// The channel sums of dw_p and dg are one: S = sum_t d n^ (times a token's gate), dw_p = b g S, dg = b w_p S.
struct BwdParams {
  const void* dy;
  const void* dres;
  const void* x;
  const __nv_bfloat16* w_post;
  const float* rstd_post;
  const void* r;
  const __nv_bfloat16* w_next;    // null: no second norm, dy is null
  const float* rstd;
  Gate gate;
  int T, H;
  float res_scale, branch_scale;
  void* dx;
  void* dresidual;
  float* dgate_token;
  float* mean;                    // [T] mean(e r^)
  float* part;                    // [P][2][H]: partial rows of dw_n and S
  int rows;                       // rows of a partial row
  unsigned int* status;
  unsigned long long timeout_ns;
  int stalled;                    // the stalled variant's: the group of every block's second row that never comes
};

// Rows of at most 8192: a block walks p.rows consecutive rows with its share of both channel sums in registers.  Rows come by
// bulk copies into a ring of shared memory, as many rows ahead as fit, in two groups with a barrier each: dy and r', which the
// first sum needs, and dres and x.  A group's place is free again once the block's sum after its last use is through, so the
// block's two barriers per row are also what the next copies wait for.
// 8192 x 6144, fp32 x, the rest bf16, a channel's gate: 128 us with the sums' kernel for 805 MB, 6.3 TB/s; 4096 x 2048, all
// fp32: 39.6 us, 5.1 TB/s, of which the start (14 rows a block) and the second kernel are what a copy does not have.  Two
// vectors a thread from 2064 columns on, so that a row is few warps and its sums few additions: 768 threads of one vector took
// 183 us, and 157 with the warps' sums read one by one and a division per mean.  At 8192 columns two rows (all fp32: one)
// fill the ring and 128 registers are not quite enough (52 to 64 bytes spilled): 2048 rows 4.1 TB/s, all fp32 5.2.
// A thread whose wait ran out goes on without its data.  What it puts in their place is NaN, which the row's sums carry to the
// other threads: nothing that depends on a row that did not come looks like a gradient, whoever reads the status.
constexpr int kBwdMaxDepth = 8, kBwdMaxWidth = 8192;
constexpr int kBwdBlocks = 2;                  // on a multiprocessor, of rows up to 2048

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Bytes of a ring place: the four rows, absent ones left out.
struct BwdShape {
  uint32_t dy, r, dres, x, row;                // offsets of a place's rows; bytes of a place
  int depth;
};

// Sum over a block of at most THREADS threads, the same in each: xor butterfly per warp, then the warps' sums, four chains of
// them.  s_part: a float per warp, 0 behind the last.  Every call is a barrier.
template <int THREADS>
__device__ __forceinline__ float row_sum(float v, float* s_part, int warp, int lane) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  if (lane == 0) s_part[warp] = v;
  __syncthreads();
  float4 s = *reinterpret_cast<const float4*>(s_part);
#pragma unroll
  for (int w = 1; w < THREADS / 128; ++w) {
    const float4 t = reinterpret_cast<const float4*>(s_part)[w];
    s.x += t.x; s.y += t.y; s.z += t.z; s.w += t.w;
  }
  return (s.x + s.y) + (s.z + s.w);
}

// V vectors of a thread, at most THREADS threads, BLOCKS of them on a multiprocessor.  STALLED: a group of the second row is
// never loaded, for a test of the time-out.
template <int V, int THREADS, int BLOCKS, bool STALLED, typename TX, typename TR, typename TD>
__global__ void __launch_bounds__(THREADS, BLOCKS) sandwich_bwd_kernel(const BwdParams p, const BwdShape sh) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(16) float s_part[2][2][32];
  __shared__ uint64_t bars[2][kBwdMaxDepth];
  __shared__ volatile int s_abort;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool next = p.w_next != nullptr, has_dres = p.dres != nullptr;
  for (int i = threadIdx.x; i < 128; i += blockDim.x) (&s_part[0][0][0])[i] = 0.0f;
  if (threadIdx.x == 0) {
    for (int i = 0; i < sh.depth; ++i) {
      mbar_init(&bars[0][i], 1);
      mbar_init(&bars[1][i], 1);
    }
    s_abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const WaitCtl wc{&s_abort, p.status, p.timeout_ns};
  const long long t0 = static_cast<long long>(blockIdx.x) * p.rows;
  const int n = static_cast<int>(min(static_cast<long long>(p.T), t0 + p.rows) - t0);
  const uint32_t bx = p.H * sizeof(TX), br = p.H * sizeof(TR), bd = p.H * sizeof(TD);
  const float inv_h = 1.0f / static_cast<float>(p.H);
  auto load = [&](int i, int at_place, int group) {   // thread 0: a group of this block's row i
    uint8_t* place = ring + at_place * sh.row;
    uint64_t* bar = &bars[group][at_place];
    const long long at = (t0 + i) * p.H;
    if (STALLED && i == 1 && group == p.stalled) return;
    if (group == 0) {
      mbar_arrive_expect_tx(bar, bd + br);
      bulk_load(place + sh.dy, static_cast<const TD*>(p.dy) + at, bd, bar);
      bulk_load(place + sh.r, static_cast<const TR*>(p.r) + at, br, bar);
    } else {
      mbar_arrive_expect_tx(bar, bx + (has_dres ? br : 0));
      if (has_dres) bulk_load(place + sh.dres, static_cast<const TR*>(p.dres) + at, br, bar);
      bulk_load(place + sh.x, static_cast<const TX*>(p.x) + at, bx, bar);
    }
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < sh.depth && i < n; ++i) {
      if (next) load(i, i, 0);
      load(i, i, 1);
    }
  }
  Raw8<__nv_bfloat16> wn[V];
  float wp[V][8];                              // w_p, times b and the gate of a channel
  float dwn[V][8], s[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * blockDim.x + threadIdx.x) * 8;
    wn[v].zero();
#pragma unroll
    for (int i = 0; i < 8; ++i) wp[v][i] = 0.0f;
    if (c < p.H) {
      if (next) wn[v].load(p.w_next + c);
      load8(p.w_post + c, wp[v]);
      if (p.gate.channel != nullptr) {
        float f[8];
        branch_factor(p.gate, p.branch_scale, 0.0f, c, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) wp[v][i] *= f[i];
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) dwn[v][i] = s[v][i] = 0.0f;
  }
  bool ok = true;
  float next_p = 0.0f, next_r = 0.0f, next_g = 1.0f;           // the row's numbers, a row ahead
  auto fetch = [&](int i) {
    next_p = __ldg(p.rstd_post + t0 + i);
    if (next) next_r = __ldg(p.rstd + t0 + i);
    if (p.gate.token != nullptr) next_g = __ldg(p.gate.token + t0 + i);
  };
  if (n > 0) fetch(0);
  int at_place = 0;
  uint32_t phase = 0;
  for (int i = 0; i < n; ++i) {
    const long long t = t0 + i;
    const uint8_t* place = ring + at_place * sh.row;
    float rstd_p = next_p, rstd = next_r, res_scale = p.res_scale;
    const float g = next_g;
    if (i + 1 < n) fetch(i + 1);
    float d[V][8];                             // e
    float n_r[V][8];
    float mean = 0.0f;
    if (next) {
      ok = ok && mbar_wait(&bars[0][at_place], phase, wc);
      if (!ok) rstd = NAN;
      float dot = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * blockDim.x + threadIdx.x) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) d[v][j] = n_r[v][j] = 0.0f;
        if (c < p.H) {
          float w[8];
          load8(reinterpret_cast<const TD*>(place + sh.dy) + c, d[v]);
          load8(reinterpret_cast<const TR*>(place + sh.r) + c, n_r[v]);
          wn[v].get(w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            n_r[v][j] *= rstd;
            dwn[v][j] = fmaf(d[v][j], n_r[v][j], dwn[v][j]);
            d[v][j] *= w[j];
            dot = fmaf(d[v][j], n_r[v][j], dot);
          }
        }
      }
      mean = row_sum<THREADS>(dot, s_part[0][i & 1], warp, lane) * inv_h;
      if (threadIdx.x == 0 && ok && i + sh.depth < n) load(i + sh.depth, at_place, 0);
    }
    ok = ok && mbar_wait(&bars[1][at_place], phase, wc);
    if (!ok) rstd_p = res_scale = NAN;
    float u[V][8], n_x[V][8];                  // u: d w_p, times the channel's gate
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * blockDim.x + threadIdx.x) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) u[v][j] = n_x[v][j] = 0.0f;
      if (c < p.H) {
        float b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = 0.0f;
        if (has_dres) load8(reinterpret_cast<const TR*>(place + sh.dres) + c, b);
        load8(reinterpret_cast<const TX*>(place + sh.x) + c, n_x[v]);
        if (next) {
#pragma unroll
          for (int j = 0; j < 8; ++j) b[j] = fmaf(rstd, fmaf(-n_r[v][j], mean, d[v][j]), b[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          n_x[v][j] *= rstd_p;
          s[v][j] = fmaf(b[j] * g, n_x[v][j], s[v][j]);
          u[v][j] = b[j] * wp[v][j];
          dot = fmaf(u[v][j], n_x[v][j], dot);
          b[j] *= res_scale;
        }
        store8(static_cast<TR*>(p.dresidual) + t * p.H + c, b);
      }
    }
    dot = row_sum<THREADS>(dot, s_part[1][i & 1], warp, lane);
    if (threadIdx.x == 0) {
      if (ok && i + sh.depth < n) load(i + sh.depth, at_place, 1);
      if (p.dgate_token != nullptr) p.dgate_token[t] = p.branch_scale * dot;
    }
    const float k = p.gate.channel != nullptr ? rstd_p : rstd_p * __fmul_rn(g, p.branch_scale);   // what u still lacks
    const float m = dot * inv_h;
    if (++at_place == sh.depth) {
      at_place = 0;
      phase ^= 1u;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * blockDim.x + threadIdx.x) * 8;
      if (c < p.H) {
#pragma unroll
        for (int j = 0; j < 8; ++j) n_x[v][j] = k * fmaf(-n_x[v][j], m, u[v][j]);
        store8(static_cast<TX*>(p.dx) + t * p.H + c, n_x[v]);
      }
    }
  }
  if (p.part != nullptr) {
    float* row = p.part + static_cast<long long>(blockIdx.x) * 2 * p.H;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * blockDim.x + threadIdx.x) * 8;
      if (c < p.H) {
        store8(row + c, dwn[v]);
        store8(row + p.H + c, s[v]);
      }
    }
  }
  if (s_abort && threadIdx.x == 0) {
    // given up: what is still on its way lands before the block exits.  Of a barrier's two parities one has passed; for the
    // other, which waits in vain where nothing was on its way, its share of the limit.
    const WaitCtl drain{nullptr, p.status, p.timeout_ns / (2 * kBwdMaxDepth)};
#pragma unroll 1
    for (int i = 0; i < 4 * sh.depth; ++i) mbar_wait_slow(&bars[i & 1][i >> 2], (i >> 1) & 1u, drain);
  }
}

// Rows above 8192, whose sums do not fit a block's registers: the rows by one kernel, the channel sums by another, which reads
// everything again (8192 x 6144 took 406 us that way, 4096 x 2048 144).
// d of 8 elements, from the row's mean(e r^).
template <typename TR, typename TD>
__device__ __forceinline__ void stream_grad(const BwdParams& p, long long at, int c, float rstd, float mean, float (&d)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) d[i] = 0.0f;
  if (p.dres != nullptr) load8(static_cast<const TR*>(p.dres) + at, d);
  if (p.w_next != nullptr) {
    float e[8], n[8], w[8];
    load8(static_cast<const TD*>(p.dy) + at, e);
    load8(static_cast<const TR*>(p.r) + at, n);
    load8(p.w_next + c, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = fmaf(rstd, fmaf(-(n[i] * rstd), mean, e[i] * w[i]), d[i]);
  }
}

// Rows: dresidual, dx, a token's dgate and mean(e r^).
template <int V, typename TX, typename TR, typename TD>
__global__ void __launch_bounds__(max_threads(V)) sandwich_bwd_rows_kernel(const BwdParams p) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s_part[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
  const long long t = blockIdx.x;
  const long long base = t * p.H;
  float rstd = 0.0f, mean = 0.0f;
  if (p.w_next != nullptr) {
    rstd = __ldg(p.rstd + t);
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * blockDim.x + threadIdx.x) * 8;
      if (c < p.H) {
        float e[8], n[8], w[8];
        load8(static_cast<const TD*>(p.dy) + base + c, e);
        load8(static_cast<const TR*>(p.r) + base + c, n);
        load8(p.w_next + c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot = fmaf(e[i] * w[i], n[i] * rstd, dot);
      }
    }
    mean = __fdiv_rn(block_sum(dot, s_part[0], warp, lane, nwarps), static_cast<float>(p.H));
    if (p.mean != nullptr && threadIdx.x == 0) p.mean[t] = mean;
  }
  const float rstd_p = __ldg(p.rstd_post + t);
  const float token = token_factor(p.gate, p.branch_scale, t);
  float u[V][8];                              // d w_p, times the channel's gate
  float dot = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * blockDim.x + threadIdx.x) * 8;
    if (c < p.H) {
      float d[8], w[8], n[8];
      stream_grad<TR, TD>(p, base + c, c, rstd, mean, d);
      load8(p.w_post + c, w);
      load8(static_cast<const TX*>(p.x) + base + c, n);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[v][i] = d[i] * w[i];
      if (p.gate.channel != nullptr) {
        float f[8];
        branch_factor(p.gate, p.branch_scale, 0.0f, c, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[v][i] *= f[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dot = fmaf(u[v][i], n[i] * rstd_p, dot);
        d[i] *= p.res_scale;
      }
      store8(static_cast<TR*>(p.dresidual) + base + c, d);
    }
  }
  dot = block_sum(dot, s_part[1], warp, lane, nwarps);
  if (p.dgate_token != nullptr && threadIdx.x == 0) p.dgate_token[t] = p.branch_scale * dot;
  const float k = p.gate.channel != nullptr ? 1.0f : token;        // what u still lacks
  const float m = __fdiv_rn(dot, static_cast<float>(p.H));
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * blockDim.x + threadIdx.x) * 8;
    if (c < p.H) {
      float n[8];
      load8(static_cast<const TX*>(p.x) + base + c, n);
#pragma unroll
      for (int i = 0; i < 8; ++i) n[i] = rstd_p * k * fmaf(-(n[i] * rstd_p), m, u[v][i]);
      store8(static_cast<TX*>(p.dx) + base + c, n);
    }
  }
}

// Columns: a thread owns 8, a block 2048, and walks p.rows consecutive rows.
template <typename TX, typename TR, typename TD>
__global__ void __launch_bounds__(256) sandwich_bwd_cols_kernel(const BwdParams p) {
  pdl_wait();
  pdl_trigger();
  const int c = (blockIdx.x * 256 + threadIdx.x) * 8;
  if (c >= p.H) return;
  const long long t0 = static_cast<long long>(blockIdx.y) * p.rows;
  const long long t1 = min(static_cast<long long>(p.T), t0 + p.rows);
  float dwn[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dwn[i] = s[i] = 0.0f;
  for (long long t = t0; t < t1; ++t) {
    const long long at = t * p.H + c;
    const float rstd_p = __ldg(p.rstd_post + t);
    float rstd = 0.0f, mean = 0.0f;
    if (p.w_next != nullptr) {
      rstd = __ldg(p.rstd + t);
      mean = p.mean[t];
      float e[8], n[8];
      load8(static_cast<const TD*>(p.dy) + at, e);
      load8(static_cast<const TR*>(p.r) + at, n);
#pragma unroll
      for (int i = 0; i < 8; ++i) dwn[i] = fmaf(e[i], n[i] * rstd, dwn[i]);
    }
    float d[8], n[8];
    stream_grad<TR, TD>(p, at, c, rstd, mean, d);
    load8(static_cast<const TX*>(p.x) + at, n);
    const float g = p.gate.token != nullptr ? __ldg(p.gate.token + t) : 1.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = fmaf(d[i] * g, n[i] * rstd_p, s[i]);
  }
  float* row = p.part + static_cast<long long>(blockIdx.y) * 2 * p.H + c;
  store8(row, dwn);
  store8(row + p.H, s);
}

// The partial rows' sums: blockIdx.y 0 is dw_n, 1 is S with what is made of it.  16 columns per block, 4 per thread: thread
// row y adds rows y, y + 64, ... ascending, the 8 thread rows of a warp fold by a xor butterfly, the 8 warps ascending.
// (Blocks of 1024 threads, which come one after the other where a row has many columns: 8192 columns 124 us instead of 120.)
constexpr int kSumCols = 16, kSumThreads = 256;
__global__ void __launch_bounds__(kSumThreads)
    sandwich_sum_kernel(const float* __restrict__ part, int P, int H, const Gate gate,
                        const __nv_bfloat16* __restrict__ w_post, float branch_scale, float* __restrict__ dw_next,
                        float* __restrict__ dw_post, float* __restrict__ dgate) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s[kSumThreads / 32][kSumCols];
  const int which = blockIdx.y;
  const int c = blockIdx.x * kSumCols + 4 * (threadIdx.x & 3);      // H is a multiple of 16
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (which == 1 || dw_next != nullptr) {
#pragma unroll 4
    for (int r = threadIdx.x >> 2; r < P; r += kSumThreads / 4) {
      const float4 a = *reinterpret_cast<const float4*>(part + (2LL * r + which) * H + c);
      v.x += a.x; v.y += a.y; v.z += a.z; v.w += a.w;
    }
  }
#pragma unroll
  for (int d = 4; d <= 16; d <<= 1) {
    v.x += __shfl_xor_sync(kFull, v.x, d);
    v.y += __shfl_xor_sync(kFull, v.y, d);
    v.z += __shfl_xor_sync(kFull, v.z, d);
    v.w += __shfl_xor_sync(kFull, v.w, d);
  }
  if ((threadIdx.x & 31) < 4) *reinterpret_cast<float4*>(&s[threadIdx.x >> 5][4 * (threadIdx.x & 3)]) = v;
  __syncthreads();
  if (threadIdx.x < kSumCols) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kSumThreads / 32; ++w) sum += s[w][threadIdx.x];
    const int h = blockIdx.x * kSumCols + threadIdx.x;
    if (which == 0) {
      if (dw_next != nullptr) dw_next[h] = sum;
    } else {
      sum *= branch_scale;
      if (gate.channel != nullptr) {
        if (dgate != nullptr) dgate[h] = sum * __bfloat162float(w_post[h]);
        sum *= __bfloat162float(gate.channel[h]);
      }
      dw_post[h] = sum;
    }
  }
}

template <typename F>
cudaError_t by_width(int H, F&& go) {
  const RowShape s = row_shape(H);
  if (s.v == 1) return go(std::integral_constant<int, 1>{}, s.threads);
  if (s.v == 2) return go(std::integral_constant<int, 2>{}, s.threads);
  return go(std::integral_constant<int, 4>{}, s.threads);
}

// Calls go with a value of the element type of each flag.
template <typename F>
cudaError_t by_types(bool a_f32, bool b_f32, F&& go) {
  if (a_f32) return b_f32 ? go(float{}, float{}) : go(float{}, __nv_bfloat16{});
  return b_f32 ? go(__nv_bfloat16{}, float{}) : go(__nv_bfloat16{}, __nv_bfloat16{});
}

Gate gate_of(const void* gate, int kind) {
  Gate g{nullptr, nullptr};
  if (kind == INVMOE_GATE_CHANNEL) g.channel = static_cast<const __nv_bfloat16*>(gate);
  if (kind == INVMOE_GATE_TOKEN) g.token = static_cast<const float*>(gate);
  return g;
}

}  // namespace

int sandwich_launch(const SandwichCall& c, cudaStream_t st) {
  ProfScope prof("sandwich_norm", st);
  const Gate gate = gate_of(c.gate, c.gate_kind);
  const cudaError_t e = by_types(c.x_f32, c.res_f32, [&](auto tx, auto tr) {
    using TX = decltype(tx);
    using TR = decltype(tr);
    return by_width(c.H, [&](auto v, int threads) {
      return launch_kernel(sandwich_kernel<v.value, TX, TR>, dim3(c.T), dim3(threads), 0, st, static_cast<const TX*>(c.x),
                           static_cast<const __nv_bfloat16*>(c.w_post), static_cast<const TR*>(c.residual), gate,
                           static_cast<const __nv_bfloat16*>(c.w_next), c.H, c.res_scale, c.branch_scale, c.eps,
                           static_cast<TR*>(c.residual_out), static_cast<__nv_bfloat16*>(c.out), static_cast<uint8_t*>(c.q),
                           c.scale, c.rstd_post, c.rstd);
    });
  });
  return check_cuda(e, "sandwich_kernel");
}

// Partial rows: a function of T and H alone, so that the order of the sums is too.  Up to 8192 columns as many blocks as are
// resident at once, with the registers and the ring that they take: two of at most 256 threads for rows up to 2048 (three:
// 42 us instead of 38.5 for 4096 x 2048), one for wider ones.
SandwichPlan sandwich_bwd_plan(int T, int H) {
  const int blocks = H <= 2048 ? 152 * kBwdBlocks : H <= kBwdMaxWidth ? 152 : 64;
  const int rows = (T - 1) / blocks + 1;
  return {rows, (T - 1) / rows + 1};
}

namespace {

template <int V, int THREADS, int BLOCKS, bool STALLED, typename TX, typename TR, typename TD>
int launch_bwd(const BwdParams& p, int threads, int parts, cudaStream_t st) {
  BwdShape sh{};
  const uint32_t bx = p.H * sizeof(TX), br = p.H * sizeof(TR), bd = p.H * sizeof(TD);   // multiples of 32
  if (p.w_next != nullptr) {
    sh.dy = 0;
    sh.r = bd;
    sh.row = bd + br;
  }
  sh.dres = sh.row;
  if (p.dres != nullptr) sh.row += br;
  sh.x = sh.row;
  sh.row += bx;
  constexpr uint32_t room = 216 * 1024 / BLOCKS;
  sh.depth = static_cast<int>(room / sh.row);
  if (sh.depth > kBwdMaxDepth) sh.depth = kBwdMaxDepth;
  if (sh.depth > p.rows) sh.depth = p.rows;
  const auto kernel = sandwich_bwd_kernel<V, THREADS, BLOCKS, STALLED, TX, TR, TD>;
  static std::atomic<uint64_t> attr_set{0};
  const int rc = set_smem_attr(reinterpret_cast<const void*>(kernel), static_cast<int>(room), attr_set);
  if (rc) return rc;
  return check_cuda(launch_kernel(kernel, dim3(parts), dim3(threads), sh.depth * sh.row, st, p, sh), "sandwich_bwd_kernel");
}

template <typename TX, typename TR, typename TD>
int launch_bwd_typed(const BwdParams& p, int parts, cudaStream_t st) {
  const int vecs = p.H / 8;
  if (vecs <= 256) return launch_bwd<1, 256, kBwdBlocks, false, TX, TR, TD>(p, (vecs + 31) / 32 * 32, parts, st);
  const int threads = (vecs + 63) / 64 * 32;
  if (vecs <= 512) return launch_bwd<2, 256, 1, false, TX, TR, TD>(p, threads, parts, st);
  if (vecs <= 768) return launch_bwd<2, 384, 1, false, TX, TR, TD>(p, threads, parts, st);
  return launch_bwd<2, 512, 1, false, TX, TR, TD>(p, threads, parts, st);
}

int launch_wide(const BwdParams& p, const SandwichBwdCall& c, int parts, cudaStream_t st) {
  {
    ProfScope prof("sandwich_bwd_rows", st);
    const int threads = row_shape(p.H).threads;
    const cudaError_t e = by_types(c.x_f32, c.res_f32, [&](auto tx, auto tr) {
      using TX = decltype(tx);
      using TR = decltype(tr);
      return c.dy_f32 ? launch_kernel(sandwich_bwd_rows_kernel<4, TX, TR, float>, dim3(p.T), dim3(threads), 0, st, p)
                      : launch_kernel(sandwich_bwd_rows_kernel<4, TX, TR, __nv_bfloat16>, dim3(p.T), dim3(threads), 0, st, p);
    });
    const int rc = check_cuda(e, "sandwich_bwd_rows_kernel");
    if (rc || p.part == nullptr) return rc;
  }
  ProfScope prof("sandwich_bwd_cols", st);
  const dim3 grid((p.H + 2047) / 2048, parts);
  const cudaError_t e = by_types(c.x_f32, c.res_f32, [&](auto tx, auto tr) {
    using TX = decltype(tx);
    using TR = decltype(tr);
    return c.dy_f32 ? launch_kernel(sandwich_bwd_cols_kernel<TX, TR, float>, grid, dim3(256), 0, st, p)
                    : launch_kernel(sandwich_bwd_cols_kernel<TX, TR, __nv_bfloat16>, grid, dim3(256), 0, st, p);
  });
  return check_cuda(e, "sandwich_bwd_cols_kernel");
}

}  // namespace

int sandwich_bwd_launch(const SandwichBwdCall& c, cudaStream_t st) {
  const SandwichPlan plan = sandwich_bwd_plan(c.T, c.H);
  BwdParams p{};
  p.dy = c.dy;
  p.dres = c.dres;
  p.x = c.x;
  p.w_post = static_cast<const __nv_bfloat16*>(c.w_post);
  p.rstd_post = c.rstd_post;
  p.r = c.r;
  p.w_next = static_cast<const __nv_bfloat16*>(c.w_next);
  p.rstd = c.rstd;
  p.gate = gate_of(c.gate, c.gate_kind);
  p.T = c.T;
  p.H = c.H;
  p.res_scale = c.res_scale;
  p.branch_scale = c.branch_scale;
  p.dx = c.dx;
  p.dresidual = c.dresidual;
  p.dgate_token = c.gate_kind == INVMOE_GATE_TOKEN ? c.dgate : nullptr;
  p.rows = plan.rows;
  p.status = c.status;
  p.timeout_ns = c.stalled_ns > 0 ? c.stalled_ns : kTimeoutNs;
  p.stalled = c.stalled;
  if (c.dw_post != nullptr) {
    p.mean = c.scratch;
    p.part = c.scratch + align_up(c.T, 64);
  }
  if (c.H <= kBwdMaxWidth) {
    ProfScope prof("sandwich_bwd", st);
    int rc = INVMOE_OK;
    if (c.stalled_ns > 0) {
      rc = launch_bwd<1, 256, kBwdBlocks, true, float, float, float>(p, (c.H / 8 + 31) / 32 * 32, plan.parts, st);
    } else {
      by_types(c.x_f32, c.res_f32, [&](auto tx, auto tr) {
        using TX = decltype(tx);
        using TR = decltype(tr);
        rc = c.dy_f32 ? launch_bwd_typed<TX, TR, float>(p, plan.parts, st)
                      : launch_bwd_typed<TX, TR, __nv_bfloat16>(p, plan.parts, st);
        return cudaSuccess;
      });
    }
    if (rc || c.dw_post == nullptr) return rc;
  } else {
    const int rc = launch_wide(p, c, plan.parts, st);
    if (rc || c.dw_post == nullptr) return rc;
  }
  ProfScope prof("sandwich_bwd_sum", st);
  return check_cuda(launch_kernel(sandwich_sum_kernel, dim3(c.H / kSumCols, 2), dim3(kSumThreads), 0, st,
                                  static_cast<const float*>(p.part), plan.parts, c.H, p.gate, p.w_post, c.branch_scale,
                                  c.w_next != nullptr ? c.dw_next : nullptr, c.dw_post,
                                  c.gate_kind == INVMOE_GATE_CHANNEL ? c.dgate : nullptr),
                    "sandwich_sum_kernel");
}

}  // namespace invmoe
