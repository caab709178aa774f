// Device helpers of the 8-bit projections.
#pragma once
#include <cuda_fp8.h>

#include "common.cuh"
#include "fp8.h"
#include "units.cuh"

namespace medusa {

// Scale of a group whose largest |x| has the bits top (as an integer: a NaN is larger than everything):
// s = 2^e with the smallest whole e >= -126 and |x| <= 448 2^e = 1.75 * 2^(e + 8), and 1/s.
struct Fp8Scale {
  float s, inv;
  bool finite;
};
__device__ __forceinline__ Fp8Scale fp8_scale(uint32_t top) {
  const int e = max((int)(top >> 23) - 135 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0), -126);   // top < 2^31
  const bool finite = top < 0x7f800000u, one = top == 0u || !finite;
  return {one ? 1.f : __uint_as_float((uint32_t)(e + 127) << 23), one ? 1.f : __uint_as_float((uint32_t)(127 - e) << 23),
          finite};
}
// Codes of four elements that have been multiplied by 1/s (nearest, ties to even).
__device__ __forceinline__ uint32_t fp8_codes(const float (&x)[4]) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}
constexpr uint32_t FP8_NANS = 0x7f7f7f7fu;
__device__ __forceinline__ void fp8_values(uint32_t codes, float (&x)[4]) {
  const float2 lo = __half22float2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xffffu), __NV_E4M3));
  const float2 hi = __half22float2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes >> 16), __NV_E4M3));
  x[0] = lo.x;
  x[1] = lo.y;
  x[2] = hi.x;
  x[3] = hi.y;
}

}  // namespace medusa
