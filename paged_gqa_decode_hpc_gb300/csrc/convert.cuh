// Conversions to the e4m3 cache type shared by the kernels that write the
// cache.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
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

// A per-tensor scale with what the fast path below needs: its reciprocal in
// fp32, and whether dividing by it is exactly multiplying by the reciprocal
// (a power of two whose reciprocal is normal).
struct E4m3Scale {
  float s, inv;
  int32_t exact;
};

inline E4m3Scale e4m3_scale(float s) {
  int e = 0;
  const bool pow2 = frexpf(s, &e) == 0.5f;
  return {s, 1.0f / s, pow2 && e > -100 && e < 100};
}

// The rare case of quantise_e4m3x8, kept out of its callers' code.
static __device__ __noinline__ uint2 quantise_e4m3x8_by_division(float4 a, float4 b, float s) {
  auto q = [s](float x) { return fabsf(x) <= 3.4028235e38f ? div_round_odd(x, s) : x; };
  return make_uint2(to_e4m3x4(make_float4(q(a.x), q(a.y), q(a.z), q(a.w))),
                    to_e4m3x4(make_float4(q(b.x), q(b.y), q(b.z), q(b.w))));
}

// e4m3(x / s) of eight values, each correctly rounded from the exact quotient,
// without dividing. y = x * (1 / s) in fp32 is within 2 ulp of the quotient, so
// both round to the same e4m3 value unless y lies within 2 ulp of the midpoint
// m of two e4m3 values: for |y| >= 2^-6 (3 mantissa bits kept) m is y with the
// lower 20 bits replaced by 2^19. There the sign of x - m s, exact in an FMA,
// tells on which side of m the quotient lies, and y becomes m or its neighbour
// on that side. (A scale of few bits puts many y there: bf16 values over
// 4 / 448 are midpoints once in 60.) Below 2^-6 all eight take the division.
__device__ __forceinline__ uint2 quantise_e4m3x8(const float (&x)[8], const E4m3Scale& sc) {
  float y[8];
  uint32_t nearest = 0xFFFFFFFFu, smallest = 0xFFFFFFFFu;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = x[i] * sc.inv;
    const uint32_t u = __float_as_uint(y[i]);
    nearest = min(nearest, (u + 0x80002u) & 0xFFFFFu);  // m -> 2
    smallest = min(smallest, 2 * u - 1);                // |y|; zero -> the largest
  }
  if (!sc.exact) {
    if (smallest < 2 * 0x3C800000u - 1)  // 0x3C800000: 2^-6
      return quantise_e4m3x8_by_division(make_float4(x[0], x[1], x[2], x[3]),
                                         make_float4(x[4], x[5], x[6], x[7]), sc.s);
    if (nearest <= 4u) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t u = __float_as_uint(y[i]), m = (u & 0xFFF00000u) | 0x80000u;
        const float r = fmaf(-__uint_as_float(m), sc.s, x[i]);
        const uint32_t side = r == 0.f ? 0u : ((__float_as_uint(r) ^ u) >> 31 ? 0xFFFFFFFFu : 1u);
        if (((u + 0x80002u) & 0xFFFFFu) <= 4u) y[i] = __uint_as_float(m + side);
      }
    }
  }
  return make_uint2(to_e4m3x4(make_float4(y[0], y[1], y[2], y[3])),
                    to_e4m3x4(make_float4(y[4], y[5], y[6], y[7])));
}

}  // namespace hpc
