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

// A per-tensor scale with what the fast path below needs: its reciprocal in fp32
// (0 where that is not a normal number), and two factors that enclose division by
// it: |x| lo <= |x| / s <= |x| hi after the rounding of the products (4 x 2^-24
// either way covers those of the factor and of the product). Both are the
// reciprocal itself for a power of two, where the product is the quotient.
struct E4m3Scale {
  float s, inv, lo, hi;
};

inline E4m3Scale e4m3_scale(float s) {
  int e = 0;
  const bool pow2 = frexpf(s, &e) == 0.5f;
  const double inv = 1.0 / (double)s, step = 4.0 / (1 << 24);
  if (!(inv >= 0x1p-120 && inv <= 0x1p120)) return {s, 0.f, 0.f, INFINITY};  // nothing enclosed
  if (pow2) return {s, (float)inv, (float)inv, (float)inv};
  return {s, (float)inv, (float)(inv * (1.0 - step)), (float)(inv * (1.0 + step))};
}

// e4m3(x / s) of eight values where some quotient lies next to the midpoint m of two
// e4m3 values. y = x * (1 / s) in fp32 is within 2 ulp of the quotient. For |y| >=
// 2^-6 (3 mantissa bits kept) m is y with the lower 20 bits replaced by 2^19, the
// sign of x - m s, exact in an FMA, tells on which side of m the quotient lies, and
// y becomes m or its neighbour on that side. What is smaller, or not finite, is
// divided. (A scale of few bits puts bf16 values here: over 4 / 448 normal ones are
// midpoints once in 134, so that six in seven warps, of 256 values each, come here.
// Of fp32 values, as turned elements are, one warp in a thousand does.)
static __device__ __noinline__ uint2 quantise_e4m3x8_near(float4 a, float4 b, float s, float inv) {
  auto q = [s, inv](float x) {
    float y = x * inv;
    const uint32_t u = __float_as_uint(y), m = (u & 0xFFF00000u) | 0x80000u;
    if (!(fabsf(y) >= 0x1p-6f && fabsf(y) < 0x1p100f))
      return fabsf(x) <= 3.4028235e38f ? div_round_odd(x, s) : x;
    if (((u + 0x80002u) & 0xFFFFFu) <= 4u) {
      const float r = fmaf(-__uint_as_float(m), s, x);
      y = __uint_as_float(m + (r == 0.f ? 0u : ((__float_as_uint(r) ^ u) >> 31 ? 0xFFFFFFFFu : 1u)));
    }
    return y;
  };
  return make_uint2(to_e4m3x4(make_float4(q(a.x), q(a.y), q(a.z), q(a.w))),
                    to_e4m3x4(make_float4(q(b.x), q(b.y), q(b.z), q(b.w))));
}

// Products of eight values with a factor, to e4m3; two products an instruction.
__device__ __forceinline__ uint2 scale_e4m3x8(const float (&x)[8], float f) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\t"
        "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(y[i]), "=f"(y[i + 1])
        : "f"(x[i]), "f"(x[i + 1]), "f"(f));
  return make_uint2(to_e4m3x4(make_float4(y[0], y[1], y[2], y[3])),
                    to_e4m3x4(make_float4(y[4], y[5], y[6], y[7])));
}

// e4m3(x / s) of eight values, each correctly rounded from the exact quotient,
// without dividing: rounding is monotone, so where the two products that enclose
// the quotient round alike, so does it.
__device__ __forceinline__ uint2 quantise_e4m3x8(const float (&x)[8], const E4m3Scale& sc) {
  const uint2 lo = scale_e4m3x8(x, sc.lo), hi = scale_e4m3x8(x, sc.hi);
  if (lo.x == hi.x && lo.y == hi.y) return lo;
  return quantise_e4m3x8_near(make_float4(x[0], x[1], x[2], x[3]),
                              make_float4(x[4], x[5], x[6], x[7]), sc.s, sc.inv);
}

}  // namespace hpc
