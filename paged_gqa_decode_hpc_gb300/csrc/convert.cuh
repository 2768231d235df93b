// Conversions to the e4m3 cache type shared by the kernels that write the
// cache.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace hpc {

// Four values to e4m3 (round to nearest even, saturating), element 0 in the
// lowest byte.
__device__ __forceinline__ uint32_t to_e4m3x4(float4 v) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v.y), "f"(v.x));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v.w), "f"(v.z));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// x / s rounded to odd in fp32: the quotient truncated toward zero, with its
// lowest mantissa bit set when the division was inexact (the FMA remainder of
// a faithfully rounded quotient is exact). A value rounded to odd with 24
// significant bits and then rounded to nearest-even at e4m3's 4 bits equals
// the nearest-even e4m3 of the exact quotient (Boldo and Melquiond, "When
// double rounding is odd", 2005: a p-bit odd rounding followed by a
// nearest rounding to at most p - 2 bits is a single correct rounding).
__device__ __forceinline__ float div_round_odd(float x, float s) {
  const float q = __fdiv_rz(x, s);
  const float r = fmaf(-q, s, x);
  return r != 0.f ? __uint_as_float(__float_as_uint(q) | 1u) : q;
}

// e4m3(v / s) of four values, each correctly rounded from the exact quotient.
__device__ __forceinline__ uint32_t quantise_e4m3x4(float4 v, float s) {
  return to_e4m3x4(make_float4(div_round_odd(v.x, s), div_round_odd(v.y, s),
                               div_round_odd(v.z, s), div_round_odd(v.w, s)));
}

}  // namespace hpc
