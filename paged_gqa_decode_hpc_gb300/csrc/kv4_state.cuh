// A softmax state of one token's 8 query heads of one KV head in a warp's lanes, as the
// 4-bit decode kernels hold, store and join it: lane (g, c) has query heads 2c and
// 2c + 1 at elements 16 g .. 16 g + 15 of the head.
#pragma once
#include <cuda_bf16.h>

#include "decode_unit.cuh"
#include "kv4.h"

namespace hpc {
namespace {

struct Kv4State {
  float m[2], l[2];    // log2 units; the sum of 2^(s - m)
  float acc[8][4];     // [element / 2][2 * (element % 2) + head]: the sum of 2^(s - m) v

  __device__ __forceinline__ void clear() {
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  }

  // dst: this lane's place of [9][32] float4
  __device__ __forceinline__ void store(float4* dst) const {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      dst[i * 32] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    dst[8 * 32] = make_float4(m[0], m[1], l[0], l[1]);
  }

  // (a state that has seen nothing, or nothing but NaN, keeps its sums)
  static __device__ __forceinline__ float factor(float from, float to) {
    return from == -INFINITY ? 1.f : ex2(from - to);
  }

  __device__ __forceinline__ void add(const Kv4State& x) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float n = fmaxf(m[e], x.m[e]);
      const float f = factor(m[e], n), a = factor(x.m[e], n);
      l[e] = l[e] * f + x.l[e] * a;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[i][e] = acc[i][e] * f + x.acc[i][e] * a;
        acc[i][2 + e] = acc[i][2 + e] * f + x.acc[i][2 + e] * a;
      }
      m[e] = n;
    }
  }

  // Joins one or two stored states (s1 may be null), both in flight together; read from
  // L2, where other SMs have written them.
  __device__ __forceinline__ void add2(const float4* s0, const float4* s1) {
    float4 x[2][9];
#pragma unroll
    for (int i = 0; i < 9; ++i) {
      x[0][i] = __ldcg(s0 + i * 32);
      x[1][i] = s1 ? __ldcg(s1 + i * 32)
                   : (i < 8 ? make_float4(0.f, 0.f, 0.f, 0.f)
                            : make_float4(-INFINITY, -INFINITY, 0.f, 0.f));
    }
    const float n0 = fmaxf(m[0], fmaxf(x[0][8].x, x[1][8].x));
    const float n1 = fmaxf(m[1], fmaxf(x[0][8].y, x[1][8].y));
    const float f0 = factor(m[0], n0), f1 = factor(m[1], n1);
    const float a0 = factor(x[0][8].x, n0), a1 = factor(x[0][8].y, n1);
    const float b0 = factor(x[1][8].x, n0), b1 = factor(x[1][8].y, n1);
    l[0] = l[0] * f0 + x[0][8].z * a0 + x[1][8].z * b0;
    l[1] = l[1] * f1 + x[0][8].w * a1 + x[1][8].w * b1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      acc[i][0] = acc[i][0] * f0 + x[0][i].x * a0 + x[1][i].x * b0;
      acc[i][1] = acc[i][1] * f1 + x[0][i].y * a1 + x[1][i].y * b1;
      acc[i][2] = acc[i][2] * f0 + x[0][i].z * a0 + x[1][i].z * b0;
      acc[i][3] = acc[i][3] * f1 + x[0][i].w * a1 + x[1][i].w * b1;
    }
    m[0] = n0;
    m[1] = n1;
  }

  // out = acc * v_scale / l and lse of token t of pair (b, h); 0 and -inf where nothing was seen
  __device__ __forceinline__ void write(const Kv4DecodeParams& p, int b, int t, int h,
                                        int lane) const {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int j = 8 * h + 2 * c + e;
      const float inv = l[e] == 0.f ? 0.f : p.v_scale / l[e];
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = pack_bf16(acc[i][e] * inv, acc[i][2 + e] * inv);
      uint4* o = reinterpret_cast<uint4*>(p.out + (int64_t)b * p.o_sb + (int64_t)t * p.o_st +
                                          (int64_t)j * p.o_sh + 16 * g);
      o[0] = make_uint4(w[0], w[1], w[2], w[3]);
      o[1] = make_uint4(w[4], w[5], w[6], w[7]);
      if (g == 0 && p.lse)
        p.lse[(int64_t)b * p.l_sb + (int64_t)t * p.l_st + (int64_t)j * p.l_sh] =
            l[e] == 0.f ? -INFINITY : (m[e] + __log2f(l[e])) * 0.6931471805599453f;
    }
  }
};

}  // namespace
}  // namespace hpc
