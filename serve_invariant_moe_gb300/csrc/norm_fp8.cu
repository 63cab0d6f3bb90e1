// norm_fp8.cu -- residual addition + RMSNorm with bf16 and/or e4m3 output, its backward, e4m3 quantisation and the
// permute of quantised rows.
//
// The norm is bound by memory: per element it reads x and the residual once and writes the new residual, the bf16 row
// and the e4m3 row once.  One block holds one row in registers between the two uses of it (sum of squares, then the
// scaled output), 8 consecutive elements per vector, so 16 lanes own one block of 128 columns and its maximum takes
// four shuffles.  The reduction order depends on H alone, never on the batch.  8192 x 6144, fp32 x, bf16 residual, both
// outputs: 83 us for 555 MB, 6.7 TB/s, what a plain copy reaches; one row: 3 us on the device, bound by the host's call.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace invmoe {

namespace {

constexpr unsigned kFull = 0xffffffffu;

// 8 consecutive elements, bf16 or fp32, as they are in memory.
template <typename T>
struct Raw8 {
  uint4 u[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) u[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if constexpr (sizeof(T) == 2) {
      const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        v[4 * i] = __uint_as_float(u[i].x);
        v[4 * i + 1] = __uint_as_float(u[i].y);
        v[4 * i + 2] = __uint_as_float(u[i].z);
        v[4 * i + 3] = __uint_as_float(u[i].w);
      }
    }
  }
};

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  Raw8<T> r;
  r.load(p);
  r.get(v);
}

__device__ __forceinline__ uint32_t bf16x2_bits(float a, float b) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&t);
}

// Stores v and replaces it by the values stored.
template <typename T>
__device__ __forceinline__ void store8(T* p, float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = bf16x2_bits(v[2 * i], v[2 * i + 1]);
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// Sum over the block, the same in every thread: xor butterfly per warp, then the warps' sums in ascending order.
__device__ __forceinline__ float block_sum(float v, float* s_part, int warp, int lane, int nwarps) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  if (nwarps == 1) return v;
  if (lane == 0) s_part[warp] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < nwarps; ++w) s += s_part[w];
  return s;
}

// e4m3 of 8 values; the 16 lanes of a block of 128 columns agree on its scale.  Lanes past the row hold zeros.
__device__ __forceinline__ void quant8(const float (&y)[8], bool in, uint8_t* q, float* scale, int lane) {
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(y[i]));
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1) a = fmaxf(a, __shfl_xor_sync(kFull, a, d));
  const float s = fp8_scale(a), inv = __frcp_rn(s);
  if (in) {
    *reinterpret_cast<uint2*>(q) = make_uint2(fp8_pack4(y[0], y[1], y[2], y[3], inv),
                                              fp8_pack4(y[4], y[5], y[6], y[7], inv));
    if ((lane & 15) == 0) *scale = s;
  }
}

// Threads of a row: one vector of 8 per thread up to H = 2048, then two up to H = 8192, then four.
struct RowShape {
  int v, threads;
};
RowShape row_shape(int H) {
  const int vecs = H / 8;
  const int v = vecs <= 256 ? 1 : vecs <= 1024 ? 2 : 4;
  return {v, ((vecs + v - 1) / v + 31) / 32 * 32};
}
constexpr int max_threads(int v) { return v == 1 ? 256 : v == 2 ? 512 : 1024; }

template <int V, typename TX, typename TR>
__global__ void __launch_bounds__(max_threads(V)) norm_kernel(const TX* __restrict__ x, const TR* res,
                                                    const __nv_bfloat16* __restrict__ weight, int H, float eps,
                                                    TR* res_out, __nv_bfloat16* __restrict__ out,
                                                    uint8_t* __restrict__ q, float* __restrict__ scale,
                                                    float* __restrict__ rstd_out) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s_part[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
  const long long t = blockIdx.x;
  const long long base = t * H;
  float r[V][8];
  float ss = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * blockDim.x + threadIdx.x) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[v][i] = 0.0f;
    if (c < H) load8(x + base + c, r[v]);
  }
  if (res != nullptr) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * blockDim.x + threadIdx.x) * 8;
      if (c < H) {
        float b[8];
        load8(res + base + c, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[v][i] = __fadd_rn(r[v][i], b[i]);
        // the norm reads the residual as it is stored: the next layer and the backward see the same row
        store8(res_out + base + c, r[v]);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(r[v][i], r[v][i], ss);
  ss = block_sum(ss, s_part, warp, lane, nwarps);
  const float rstd = __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(ss, static_cast<float>(H)), eps)));
  if (rstd_out != nullptr && threadIdx.x == 0) rstd_out[t] = rstd;
  const int nb = (H + kFp8Block - 1) / kFp8Block;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * blockDim.x + threadIdx.x) * 8;
    const bool in = c < H;
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0.0f;
    if (in) load8(weight + c, w);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = in ? __fmul_rn(__fmul_rn(r[v][i], rstd), w[i]) : 0.0f;
    if (q != nullptr) quant8(y, in, q + base + c, scale + t * nb + c / kFp8Block, lane);
    if (out != nullptr && in) store8(out + base + c, y);
  }
}

// Backward: g = dy * w, n = r * rstd, dr = rstd * (g - n * mean(g n)) + dres; dw = sum_t dy n.  A block walks
// rows_per_block consecutive rows and keeps its share of dw in registers; the partial rows are summed in order by
// dweight_kernel, so no atomics and one order for a given T and H.  4096 x 2048, fp32 dy, bf16 x and dres: 18.8 us a
// call for 84 MB, 4.5 TB/s, of which this kernel takes 13 and dweight_kernel 4; what is left over a copy is the start (nine
// rows a block) and the second kernel.  Narrow rows leave a block one or two warps and one row in flight, so they are bound
// by latency, not by memory (cold, 8192 rows of 128: 21 us, 0.4 TB/s; of 512: 23 us, 1.5 TB/s).
template <int V, typename TX, typename TD>
__global__ void __launch_bounds__(max_threads(V)) norm_bwd_kernel(const TD* __restrict__ dy, const TX* __restrict__ x,
                                                        const __nv_bfloat16* __restrict__ weight,
                                                        const float* __restrict__ rstd, const TX* dres, int T, int H,
                                                        int rows_per_block, TX* dx, float* __restrict__ dw_part) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s_part[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
  // Up to two vectors a thread keeps the row in registers and loads the next one while this one is worked on.  With four
  // (H > 8192, 1024 threads of 64 registers) only dw stays there and the row is read a second time, from L1 or L2.
  constexpr bool KEEP = V < 4;
  float w[KEEP ? V : 1][8], dw[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * blockDim.x + threadIdx.x) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[v][i] = 0.0f;
    if constexpr (KEEP) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[v][i] = 0.0f;
      if (c < H) load8(weight + c, w[v]);
    }
  }
  const long long t0 = static_cast<long long>(blockIdx.x) * rows_per_block;
  const long long t1 = min(static_cast<long long>(T), t0 + rows_per_block);
  int buf = 0;
  if constexpr (KEEP) {
    Raw8<TD> next_dy[V];
    Raw8<TX> next_x[V], next_res[V];
    float next_rs = 0.0f;
    auto fetch = [&](long long t) {
      next_rs = __ldg(rstd + t);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * blockDim.x + threadIdx.x) * 8;
        next_dy[v].zero();
        next_x[v].zero();
        next_res[v].zero();
        if (c < H) {
          next_dy[v].load(dy + t * H + c);
          next_x[v].load(x + t * H + c);
          if (dres != nullptr) next_res[v].load(dres + t * H + c);
        }
      }
    };
    if (t0 < t1) fetch(t0);
    for (long long t = t0; t < t1; ++t) {
      const float rs = next_rs;
      float g[V][8], n[V][8];
      Raw8<TX> res[V];
      float dot = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        next_dy[v].get(g[v]);
        next_x[v].get(n[v]);
        res[v] = next_res[v];
      }
      if (t + 1 < t1) fetch(t + 1);
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          n[v][i] *= rs;
          dw[v][i] = fmaf(g[v][i], n[v][i], dw[v][i]);
          g[v][i] *= w[v][i];
          dot = fmaf(g[v][i], n[v][i], dot);
        }
      dot = block_sum(dot, s_part[buf], warp, lane, nwarps);   // two buffers: one barrier per row
      buf ^= 1;
      const float mean = __fdiv_rn(dot, static_cast<float>(H));
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * blockDim.x + threadIdx.x) * 8;
        if (c < H) {
          float d[8], b[8];
          res[v].get(b);                                       // zeros without dres
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] = rs * (g[v][i] - n[v][i] * mean) + b[i];
          store8(dx + t * H + c, d);
        }
      }
    }
  } else {
    for (long long t = t0; t < t1; ++t) {
      const float rs = __ldg(rstd + t);
      float dot = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * blockDim.x + threadIdx.x) * 8;
        if (c < H) {
          float g[8], n[8], wv[8];
          load8(dy + t * H + c, g);
          load8(x + t * H + c, n);
          load8(weight + c, wv);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            n[i] *= rs;
            dw[v][i] = fmaf(g[i], n[i], dw[v][i]);
            g[i] *= wv[i];
            dot = fmaf(g[i], n[i], dot);
          }
        }
      }
      dot = block_sum(dot, s_part[buf], warp, lane, nwarps);
      buf ^= 1;
      const float mean = __fdiv_rn(dot, static_cast<float>(H));
#pragma unroll 1
      for (int v = 0; v < V; ++v) {
        const int c = (v * blockDim.x + threadIdx.x) * 8;
        if (c < H) {
          float d[8], b[8], n[8], wv[8];
          load8(dy + t * H + c, d);
          load8(x + t * H + c, n);
          load8(weight + c, wv);
#pragma unroll
          for (int i = 0; i < 8; ++i) b[i] = 0.0f;
          if (dres != nullptr) load8(dres + t * H + c, b);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            n[i] *= rs;
            d[i] *= wv[i];
            d[i] = rs * (d[i] - n[i] * mean) + b[i];
          }
          store8(dx + t * H + c, d);
        }
      }
    }
  }
  if (dw_part != nullptr) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * blockDim.x + threadIdx.x) * 8;
      if (c < H) store8(dw_part + static_cast<long long>(blockIdx.x) * H + c, dw[v]);
    }
  }
}

// dw[h] = sum over P partial rows, 16 columns per block (so that a 2048-wide row gives 128 blocks), 4 per thread: thread row
// y adds rows y, y + 256, ... ascending; the 8 thread rows of a warp fold by a xor butterfly; the 32 warps ascending.
constexpr int kDwCols = 16, kDwThreads = 1024;
__global__ void __launch_bounds__(kDwThreads) dweight_kernel(const float* __restrict__ part, int P, int H,
                                                             float* __restrict__ dw) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s[32][kDwCols];
  const int c = blockIdx.x * kDwCols + 4 * (threadIdx.x & 3);      // H is a multiple of 16
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int r = threadIdx.x >> 2; r < P; r += kDwThreads / 4) {
    const float4 a = *reinterpret_cast<const float4*>(part + static_cast<long long>(r) * H + c);
    v.x += a.x; v.y += a.y; v.z += a.z; v.w += a.w;
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
  if (threadIdx.x < kDwCols) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < 32; ++w) sum += s[w][threadIdx.x];
    dw[blockIdx.x * kDwCols + threadIdx.x] = sum;
  }
}

// e4m3 of row-major [rows, cols] with a scale per row and 128 columns: 16 lanes per block, 2 blocks per warp.
template <typename TX>
__global__ void __launch_bounds__(256) quant_rows_kernel(const TX* __restrict__ x, long long rows, int cols, int nb,
                                                         uint8_t* __restrict__ q, float* __restrict__ scale) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long total = rows * nb;
  const long long step = static_cast<long long>(gridDim.x) * (blockDim.x / 16);
  // both halves of a warp make the same number of turns: the loop runs on the warp's first block
  for (long long b0 = (static_cast<long long>(blockIdx.x) * blockDim.x + (threadIdx.x & ~31)) / 16; b0 < total;
       b0 += step) {
    const long long b = b0 + (lane >> 4);
    const long long r = b / nb;
    const int c = static_cast<int>(b - r * nb) * kFp8Block + (lane & 15) * 8;
    const bool in = b < total && c < cols;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = 0.0f;
    if (in) load8(x + r * cols + c, y);
    quant8(y, in, q + r * cols + c, scale + b, lane);
  }
}

// e4m3 of [rows, cols] with a scale per 128 x 128 block: one thread block of 256 per block, 8 elements x 8 rows each.
template <typename TX>
__global__ void __launch_bounds__(256) quant_blocks_kernel(const TX* __restrict__ x, int rows, int cols, int nb,
                                                           int rb, uint8_t* __restrict__ q, float* __restrict__ scale) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s_max[8];
  const long long bank = blockIdx.x / (static_cast<long long>(nb) * rb);
  const int in_bank = static_cast<int>(blockIdx.x - bank * nb * rb);
  const int br = in_bank / nb, bc = in_bank - br * nb;
  const int c = bc * kFp8Block + (threadIdx.x & 15) * 8;
  const long long first = bank * rows + static_cast<long long>(br) * kFp8Block;
  const int n_rows = min(kFp8Block, rows - br * kFp8Block);
  float y[8][8];
  float a = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int r = j * 16 + (threadIdx.x >> 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[j][i] = 0.0f;
    if (r < n_rows && c < cols) load8(x + (first + r) * cols + c, y[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(y[j][i]));
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) a = fmaxf(a, __shfl_xor_sync(kFull, a, d));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) a = fmaxf(a, s_max[w]);
  const float s = fp8_scale(a), inv = __frcp_rn(s);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int r = j * 16 + (threadIdx.x >> 4);
    if (r < n_rows && c < cols)
      *reinterpret_cast<uint2*>(q + (first + r) * cols + c) =
          make_uint2(fp8_pack4(y[j][0], y[j][1], y[j][2], y[j][3], inv),
                     fp8_pack4(y[j][4], y[j][5], y[j][6], y[j][7], inv));
  }
  if (threadIdx.x == 0) scale[blockIdx.x] = s;
}

// xp[slot_row[t, j]] = x[t] for e4m3 rows (16-byte vectors) and their scales: one warp per token, each row read once.
__global__ void __launch_bounds__(256) permute_fp8_kernel(const uint4* __restrict__ q, const float* __restrict__ scale,
                                                          const int32_t* __restrict__ slot_row, long long T, int k,
                                                          int vec, int nb, uint4* __restrict__ xp,
                                                          float* __restrict__ xp_scale) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  // a warp copies segment `seg` (64 vectors) of token t; segment 0 also copies the scales
  const int nseg = (vec + 63) / 64;
  const long long items = T * nseg;
  for (long long it = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); it < items;
       it += static_cast<long long>(gridDim.x) * 8) {
    const long long t = it / nseg;
    const int seg = static_cast<int>(it - t * nseg);
    const int my_row = lane < k ? __ldg(slot_row + t * k + lane) : 0;
    const int c0 = seg * 64 + lane, c1 = c0 + 32;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const uint4 v0 = c0 < vec ? __ldg(q + t * vec + c0) : zero;
    const uint4 v1 = c1 < vec ? __ldg(q + t * vec + c1) : zero;
    for (int j = 0; j < k; ++j) {
      const long long row = __shfl_sync(kFull, my_row, j);
      if (c0 < vec) xp[row * vec + c0] = v0;
      if (c1 < vec) xp[row * vec + c1] = v1;
    }
    if (seg == 0)
      for (int c = lane; c < nb; c += 32) {
        const float s = __ldg(scale + t * nb + c);
        for (int j = 0; j < k; ++j) xp_scale[static_cast<long long>(__ldg(slot_row + t * k + j)) * nb + c] = s;
      }
  }
}

template <typename TX, typename TR>
cudaError_t norm_typed(const void* x, const void* res, const void* weight, int T, int H, float eps, void* res_out,
                       void* out, void* q, float* scale, float* rstd, cudaStream_t st) {
  const RowShape s = row_shape(H);
  auto go = [&](auto kernel) {
    return launch_kernel(kernel, dim3(T), dim3(s.threads), 0, st, static_cast<const TX*>(x),
                         static_cast<const TR*>(res), static_cast<const __nv_bfloat16*>(weight), H, eps,
                         static_cast<TR*>(res_out), static_cast<__nv_bfloat16*>(out), static_cast<uint8_t*>(q), scale,
                         rstd);
  };
  if (s.v == 1) return go(norm_kernel<1, TX, TR>);
  if (s.v == 2) return go(norm_kernel<2, TX, TR>);
  return go(norm_kernel<4, TX, TR>);
}

template <typename TX, typename TD>
cudaError_t norm_bwd_typed(const void* dy, const void* x, const void* weight, const float* rstd, const void* dres,
                           int T, int H, int rows, int P, void* dx, float* part, cudaStream_t st) {
  const RowShape s = row_shape(H);
  auto go = [&](auto kernel) {
    return launch_kernel(kernel, dim3(P), dim3(s.threads), 0, st, static_cast<const TD*>(dy),
                         static_cast<const TX*>(x), static_cast<const __nv_bfloat16*>(weight), rstd,
                         static_cast<const TX*>(dres), T, H, rows, static_cast<TX*>(dx), part);
  };
  if (s.v == 1) return go(norm_bwd_kernel<1, TX, TD>);
  if (s.v == 2) return go(norm_bwd_kernel<2, TX, TD>);
  return go(norm_bwd_kernel<4, TX, TD>);
}

}  // namespace

int norm_launch(const void* x, int x_f32, const void* res, int res_f32, const void* weight, int T, int H, float eps,
                void* res_out, void* out, void* q, float* scale, float* rstd, cudaStream_t st) {
  ProfScope prof("add_rms_norm", st);
  cudaError_t e;
  if (x_f32)
    e = res_f32 ? norm_typed<float, float>(x, res, weight, T, H, eps, res_out, out, q, scale, rstd, st)
                : norm_typed<float, __nv_bfloat16>(x, res, weight, T, H, eps, res_out, out, q, scale, rstd, st);
  else
    e = res_f32 ? norm_typed<__nv_bfloat16, float>(x, res, weight, T, H, eps, res_out, out, q, scale, rstd, st)
                : norm_typed<__nv_bfloat16, __nv_bfloat16>(x, res, weight, T, H, eps, res_out, out, q, scale, rstd, st);
  return check_cuda(e, "norm_kernel");
}

// Rows of one block, and so of one partial row of dw: as many blocks as are resident at once for rows of 2048 and more,
// three of 256 threads to an SM, two where a thread has two vectors, one of more threads (narrower rows, of which more
// blocks would fit, take the 456 too).  More blocks write more partial rows and leave a partly filled wave (1000 x 6144,
// both kernels: 18 us with 456 blocks, 12.6 with 152), fewer leave registers idle (4096 x 2048, norm_bwd_kernel alone: 13 us
// with 456, 17 with 304; 8192 x 4096: 56 with 456, 48 with 304, 66 with 152).  A function of T and H alone, not of the
// device, so that the order of the sum is too.
int norm_bwd_rows(int T, int H) {
  const RowShape s = row_shape(H);
  const int blocks = s.v == 1 ? 456 : s.threads <= 256 ? 304 : 152;
  return (T - 1) / blocks + 1;
}

int norm_bwd_launch(const void* dy, int dy_f32, const void* x, int x_f32, const void* weight, const float* rstd,
                    const void* dres, int T, int H, void* dx, float* dw, float* part, cudaStream_t st) {
  const int rows = norm_bwd_rows(T, H), P = (T - 1) / rows + 1;
  {
    ProfScope prof("rms_norm_bwd", st);
    cudaError_t e;
    float* pp = dw != nullptr ? part : nullptr;
    if (x_f32)
      e = dy_f32 ? norm_bwd_typed<float, float>(dy, x, weight, rstd, dres, T, H, rows, P, dx, pp, st)
                 : norm_bwd_typed<float, __nv_bfloat16>(dy, x, weight, rstd, dres, T, H, rows, P, dx, pp, st);
    else
      e = dy_f32 ? norm_bwd_typed<__nv_bfloat16, float>(dy, x, weight, rstd, dres, T, H, rows, P, dx, pp, st)
                 : norm_bwd_typed<__nv_bfloat16, __nv_bfloat16>(dy, x, weight, rstd, dres, T, H, rows, P, dx, pp, st);
    const int rc = check_cuda(e, "norm_bwd_kernel");
    if (rc || dw == nullptr) return rc;
  }
  ProfScope prof("rms_norm_dweight", st);
  return check_cuda(launch_kernel(dweight_kernel, dim3(H / kDwCols), dim3(kDwThreads), 0, st,
                                  static_cast<const float*>(part), P, H, dw),
                    "dweight_kernel");
}

int quantize_launch(const void* x, int x_f32, long long banks, int rows, int cols, int block_rows, void* q,
                    float* scale, cudaStream_t st) {
  const int nb = (cols + kFp8Block - 1) / kFp8Block;
  uint8_t* qq = static_cast<uint8_t*>(q);
  ProfScope prof("fp8_quantize", st);
  if (block_rows == 1) {
    const long long total = banks * rows;
    const long long want = (total * nb + 15) / 16;
    int sms = 0;
    const int rc = device_sm_count(&sms);
    if (rc) return rc;
    const dim3 g(static_cast<unsigned>(want < sms * 16LL ? want : sms * 16LL));
    return check_cuda(x_f32 ? launch_kernel(quant_rows_kernel<float>, g, dim3(256), 0, st, static_cast<const float*>(x),
                                            total, cols, nb, qq, scale)
                            : launch_kernel(quant_rows_kernel<__nv_bfloat16>, g, dim3(256), 0, st,
                                            static_cast<const __nv_bfloat16*>(x), total, cols, nb, qq, scale),
                      "quant_rows_kernel");
  }
  const int rb = (rows - 1) / kFp8Block + 1;
  const long long blocks = banks * rb * nb;
  if (blocks > 0x7fffffffLL) return set_error(INVMOE_ERR_UNSUPPORTED_SHAPE, "too many blocks for one launch");
  const dim3 g(static_cast<unsigned>(blocks));
  return check_cuda(x_f32 ? launch_kernel(quant_blocks_kernel<float>, g, dim3(256), 0, st, static_cast<const float*>(x),
                                          rows, cols, nb, rb, qq, scale)
                          : launch_kernel(quant_blocks_kernel<__nv_bfloat16>, g, dim3(256), 0, st,
                                          static_cast<const __nv_bfloat16*>(x), rows, cols, nb, rb, qq, scale),
                    "quant_blocks_kernel");
}

int permute_fp8_launch(const void* q, const float* scale, const int32_t* slot_row, int T, int k, int H, void* xp,
                       float* xp_scale, cudaStream_t st) {
  const int vec = H / 16, nb = (H + kFp8Block - 1) / kFp8Block;
  int sms = 0;
  const int rc = device_sm_count(&sms);
  if (rc) return rc;
  const long long want = (static_cast<long long>(T) * ((vec + 63) / 64) + 7) / 8;
  const dim3 g(static_cast<unsigned>(want < sms * 8LL ? want : sms * 8LL));
  ProfScope prof("permute_fp8", st);
  return check_cuda(launch_kernel(permute_fp8_kernel, g, dim3(256), 0, st, static_cast<const uint4*>(q), scale,
                                  slot_row, static_cast<long long>(T), k, vec, nb, static_cast<uint4*>(xp), xp_scale),
                    "permute_fp8_kernel");
}

}  // namespace invmoe
