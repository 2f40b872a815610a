// Device arithmetic of the e4m3 quantisers: a block's power-of-two scale and
// the rounding of four values.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace lmoe {

// max(m, |f|), f left out when it is not finite.
__device__ __forceinline__ float finite_max(float m, float f) {
  const float a = fabsf(f);
  return a < INFINITY ? fmaxf(m, a) : m;
}
// The smallest e in [-126, 127] with amax <= 448 * 2^e; 0 for amax = 0.
// 448 = 1.75 * 2^8: with amax = m 2^p, 1 <= m < 2, e is p - 8, one more when
// m > 1.75.  (A subnormal amax has p below any normal one's and ends at -126.)
__device__ __forceinline__ int scale_exponent(float amax) {
  if (amax == 0.0f) return 0;
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, -126);
}
__device__ __forceinline__ float pow2_f(int e) {  // -126 <= e <= 127
  return __uint_as_float((uint32_t)(e + 127) << 23);
}
// Four e4m3 values of finite numbers or NaN, the first in the lowest byte.
__device__ __forceinline__ uint32_t pack_e4m3_finite(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
// Four e4m3 values, the first in the lowest byte; NaN and infinities give NaN.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  const float z = 0.0f;  // x + (x * 0): NaN for an infinity, x otherwise
  return pack_e4m3_finite(a + a * z, b + b * z, c + c * z, d + d * z);
}

}  // namespace lmoe
