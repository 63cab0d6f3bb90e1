// sandwich_norm.cu -- the norms after and before a block in one pass, and their backward.
//
//   n = x rstd_p w_p,  r' = a r + b g n  (stored in the residual's type),  y = r' rstd w_n
//
// with rstd_p = 1 / sqrt(mean(x^2) + eps) of the block's output x, rstd likewise of the stored row r', a and b scalars and
// the gate g one number per channel or per token (or absent).  Bound by memory: per element the forward reads x and r and
// writes r' and y.  One block holds one row in registers across both sums; the reduction orders depend on H alone.
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

template <int V, typename TX, typename TR>
__global__ void __launch_bounds__(max_threads(V))
    sandwich_kernel(const TX* __restrict__ x, const __nv_bfloat16* __restrict__ w_post, const TR* res, const Gate gate,
                    const __nv_bfloat16* __restrict__ w_next, int H, float res_scale, float branch_scale, float eps,
                    TR* res_out, __nv_bfloat16* __restrict__ out, uint8_t* __restrict__ q, float* __restrict__ scale,
                    float* __restrict__ rstd_post, float* __restrict__ rstd_out) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s_part[2][32];
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
  const float rstd_p = inv_rms(block_sum(ss, s_part[0], warp, lane, nwarps), H, eps);
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
  const float rstd = inv_rms(block_sum(ss, s_part[1], warp, lane, nwarps), H, eps);
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
};

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
// row y adds rows y, y + 256, ... ascending, the 8 thread rows of a warp fold by a xor butterfly, the 32 warps ascending.
constexpr int kSumCols = 16, kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads)
    sandwich_sum_kernel(const float* __restrict__ part, int P, int H, const Gate gate,
                        const __nv_bfloat16* __restrict__ w_post, float branch_scale, float* __restrict__ dw_next,
                        float* __restrict__ dw_post, float* __restrict__ dgate) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s[32][kSumCols];
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
    for (int w = 0; w < 32; ++w) sum += s[w][threadIdx.x];
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

// Partial rows: a function of T and H alone, so that the order of the sums is too.
SandwichPlan sandwich_bwd_plan(int T, int H) {
  (void)H;
  const int rows = (T - 1) / 64 + 1;
  return {rows, (T - 1) / rows + 1};
}

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
  if (c.dw_post != nullptr) {
    p.mean = c.scratch;
    p.part = c.scratch + align_up(c.T, 64);
  }
  {
    ProfScope prof("sandwich_bwd_rows", st);
    const cudaError_t e = by_types(c.x_f32, c.res_f32, [&](auto tx, auto tr) {
      using TX = decltype(tx);
      using TR = decltype(tr);
      return by_width(c.H, [&](auto v, int threads) {
        return c.dy_f32 ? launch_kernel(sandwich_bwd_rows_kernel<v.value, TX, TR, float>, dim3(c.T), dim3(threads), 0, st, p)
                        : launch_kernel(sandwich_bwd_rows_kernel<v.value, TX, TR, __nv_bfloat16>, dim3(c.T), dim3(threads),
                                        0, st, p);
      });
    });
    const int rc = check_cuda(e, "sandwich_bwd_rows_kernel");
    if (rc || c.dw_post == nullptr) return rc;
  }
  {
    ProfScope prof("sandwich_bwd_cols", st);
    const dim3 grid((c.H + 2047) / 2048, plan.parts);
    const cudaError_t e = by_types(c.x_f32, c.res_f32, [&](auto tx, auto tr) {
      using TX = decltype(tx);
      using TR = decltype(tr);
      return c.dy_f32 ? launch_kernel(sandwich_bwd_cols_kernel<TX, TR, float>, grid, dim3(256), 0, st, p)
                      : launch_kernel(sandwich_bwd_cols_kernel<TX, TR, __nv_bfloat16>, grid, dim3(256), 0, st, p);
    });
    const int rc = check_cuda(e, "sandwich_bwd_cols_kernel");
    if (rc) return rc;
  }
  ProfScope prof("sandwich_bwd_sum", st);
  return check_cuda(launch_kernel(sandwich_sum_kernel, dim3(c.H / kSumCols, 2), dim3(kSumThreads), 0, st,
                                  static_cast<const float*>(p.part), plan.parts, c.H, p.gate, p.w_post, c.branch_scale,
                                  c.w_next != nullptr ? c.dw_next : nullptr, c.dw_post,
                                  c.gate_kind == INVMOE_GATE_CHANNEL ? c.dgate : nullptr),
                    "sandwich_sum_kernel");
}

}  // namespace invmoe
