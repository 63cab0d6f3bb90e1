// row_ops.cuh -- what the row kernels (norms, quantisation) share: vectors of 8 elements, the block's sum, e4m3 of a vector,
// threads per row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8.cuh"

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

}  // namespace

}  // namespace invmoe
