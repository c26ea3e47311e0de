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

// int8 code of a quotient: rounded to the nearest integer with ties to even, clamped to
// [-127, 127]; NaN gives 0.  int8_code: of x / scale, a correctly rounded fp32 division.
__device__ __forceinline__ int int8_code_of(float q) {
  const int c = __float2int_rn(q);  // saturates at the int range for +-inf
  return q != q ? 0 : (c < -127 ? -127 : (c > 127 ? 127 : c));
}
__device__ __forceinline__ int int8_code(float x, float scale) {
  return int8_code_of(__fdiv_rn(x, scale));
}

// Many quotients by one scale, correctly rounded: with r the correctly rounded reciprocal
// and q0 = RN(x r), RN(q0 + r RN(x - q0 scale)) is RN(x / scale) (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990), three operations in
// place of a division each.  A q0 beyond any code's range is cut off first, so that the
// remainder of an infinity stays one; quotients so small that the remainder could
// underflow are coded 0 either way.  Scales of extreme magnitude are divided by.  (Beside the
// theorem: for every 24-bit scale, the five dividends nearest to every border of the codes
// give the quotients that a division gives.)
struct Quotients {
  float scale, r;
  bool divides;
  __device__ __forceinline__ float operator()(float x) const {
    if (divides) return __fdiv_rn(x, scale);
    const float q = fminf(fmaxf(x * r, -1024.f), 1024.f);
    return x == 0.f ? q : fmaf(fmaf(-q, scale, x), r, q);  // a zero keeps its sign
  }
};

__device__ __forceinline__ Quotients quotients_by(float s) {
  return Quotients{s, __fdiv_rn(1.f, s), !(s >= 0x1p-60f && s <= 0x1p60f)};
}

// E4M3 codes of two quotients, the first in the low byte (saturated; NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3_codes(float q0, float q1) {
  return __nv_cvt_float2_to_fp8x2(make_float2(q0, q1), __NV_SATFINITE, __NV_E4M3);
}

}  // namespace pkv
