// fp8.cuh -- e4m3 conversion and block scales shared by the 8-bit kernels (sm_103a).
#pragma once

#include <cuda_fp8.h>
#include <cstdint>

namespace invmoe {

constexpr int kFp8Block = 128;            // columns (and, for weights, rows) that share one scale
constexpr float kFp8Max = 448.0f;         // largest finite e4m3 value
constexpr float kFp8MinScale = 1.17549435e-38f;   // 2^-126: a block of zeros keeps a normal scale

// scale = max(amax / 448, 2^-126).  Dividing (not multiplying by a rounded 1/448) and taking the reciprocal
// of the rounded scale afterwards makes both steps correctly rounded, so that any other correctly rounded
// implementation of the same two steps gets the same bits.  fmaxf drops a NaN; amax itself ignores NaN
// elements, which become e4m3 NaNs on their own, while an infinite amax gives an infinite scale and turns the
// block's infinite elements into NaN.
__device__ __forceinline__ float fp8_scale(float amax) { return fmaxf(__fdiv_rn(amax, kFp8Max), kFp8MinScale); }

// Four values, scaled by `inv`, rounded to nearest even, clipped to +-448; value 0 in the lowest byte.
__device__ __forceinline__ uint32_t fp8_pack4(float v0, float v1, float v2, float v3, float inv) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(v0, inv), __fmul_rn(v1, inv)), __NV_SATFINITE,
                                               __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(v2, inv), __fmul_rn(v3, inv)), __NV_SATFINITE,
                                               __NV_E4M3);
  return lo | (hi << 16);
}

__device__ __forceinline__ uint8_t fp8_one(float v, float inv) {
  return static_cast<uint8_t>(__nv_cvt_float_to_fp8(__fmul_rn(v, inv), __NV_SATFINITE, __NV_E4M3));
}

}  // namespace invmoe
