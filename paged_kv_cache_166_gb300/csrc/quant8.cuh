// The 8-bit cache formats' element arithmetic, shared by the kernels that write them.
#pragma once

#include <cuda_fp8.h>

#include <cstdint>

namespace pkv {

// Byte of token t (0..15) inside a 16-byte head_dim row of an 8-bit V tile: the
// tokens are stored in the order 0 1 8 9 2 3 10 11 4 5 12 13 6 7 14 15.
__device__ __forceinline__ int fp8_v_pos(int t) {
  return t < 8 ? 4 * (t >> 1) + (t & 1) : 4 * ((t - 8) >> 1) + 2 + (t & 1);
}

// E4M3 code of x / scale: the quotient a correctly rounded fp32 division, then round
// to nearest even with saturation to +-448 (the hardware conversion); NaN stays NaN.
__device__ __forceinline__ uint8_t e4m3_code(float x, float scale) {
  return __nv_cvt_float_to_fp8(__fdiv_rn(x, scale), __NV_SATFINITE, __NV_E4M3);
}

// int8 code of x / scale: the quotient a correctly rounded fp32 division, rounded to
// the nearest integer with ties to even, clamped to [-127, 127]; NaN gives 0.
__device__ __forceinline__ int int8_code(float x, float scale) {
  const float q = __fdiv_rn(x, scale);
  const int c = __float2int_rn(q);  // saturates at the int range for +-inf
  return q != q ? 0 : (c < -127 ? -127 : (c > 127 ? 127 : c));
}

}  // namespace pkv
