// A quarter of a softmax state, as the 4-bit decode kernel stores and joins it. A state is
// one token's 8 query heads of one KV head in a warp's lanes: lane (g, c) has query heads
// 2c and 2c + 1 at elements 16 g .. 16 g + 15 of the head, as eight slices of two elements,
// and both heads' maximum and sum. Quarter e is slices 2e and 2e + 1. Stored, a state is
// [9][32] float4: slice i of each lane as (element, head) = (0, 0), (0, 1), (1, 0), (1, 1),
// then (m, m, l, l).
#pragma once
#include <cuda_bf16.h>

#include "decode_unit.cuh"
#include "kv4.h"

namespace hpc {
namespace {

struct Kv4Slices {
  float m[2], l[2];  // log2 units; the sum of 2^(s - m)
  float acc[2][4];   // the sum of 2^(s - m) v

  __device__ __forceinline__ void clear() {
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  }

  // (a state that has seen nothing, or nothing but NaN, keeps its sums)
  static __device__ __forceinline__ float factor(float from, float to) {
    return from == -INFINITY ? 1.f : ex2(from - to);
  }

  // dst: this lane's place in a stored state; the first quarter brings m and l
  __device__ __forceinline__ void store(float4* dst, int e) const {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      dst[(2 * e + i) * 32] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    if (e == 0) dst[8 * 32] = make_float4(m[0], m[1], l[0], l[1]);
  }

  // Joins the same quarter of N other states (m, l, slice 0, slice 1 each).
  template <int N>
  __device__ __forceinline__ void add(const float4 (&ml)[N], const float4 (&x)[N][2]) {
    float n0 = m[0], n1 = m[1];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      n0 = fmaxf(n0, ml[k].x);
      n1 = fmaxf(n1, ml[k].y);
    }
    const float f0 = factor(m[0], n0), f1 = factor(m[1], n1);
    m[0] = n0;
    m[1] = n1;
    l[0] *= f0;
    l[1] *= f1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      acc[i][0] *= f0;
      acc[i][1] *= f1;
      acc[i][2] *= f0;
      acc[i][3] *= f1;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float w0 = factor(ml[k].x, n0), w1 = factor(ml[k].y, n1);
      l[0] += ml[k].z * w0;
      l[1] += ml[k].w * w1;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        acc[i][0] += x[k][i].x * w0;
        acc[i][1] += x[k][i].y * w1;
        acc[i][2] += x[k][i].z * w0;
        acc[i][3] += x[k][i].w * w1;
      }
    }
  }

  // Joins n stored states, four in flight together; place(i): this lane's place in the
  // i-th. Read from L2, where other SMs have written them.
  template <typename F>
  __device__ __forceinline__ void join(int n, int e, F place) {
    constexpr int N = 4;
#pragma unroll 1
    for (int i = 0; i < n; i += N) {
      float4 ml[N], x[N][2];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        ml[k] = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
        x[k][0] = x[k][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i + k < n) {
          const float4* s = place(i + k);
          ml[k] = __ldcg(s + 8 * 32);
          x[k][0] = __ldcg(s + (2 * e) * 32);
          x[k][1] = __ldcg(s + (2 * e + 1) * 32);
        }
      }
      add(ml, x);
    }
  }

  // out = acc * v_scale / l and lse of pair (b, h); 0 and -inf where nothing was seen
  __device__ __forceinline__ void write(const Kv4DecodeParams& p, int b, int h, int e, int lane) const {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int j = 8 * h + 2 * c + x;
      const float inv = l[x] == 0.f ? 0.f : p.v_scale / l[x];
      uint2* o = reinterpret_cast<uint2*>(p.out + (int64_t)b * p.o_sb + (int64_t)j * p.o_sh +
                                          16 * g + 4 * e);
      *o = make_uint2(pack_bf16(acc[0][x] * inv, acc[0][2 + x] * inv),
                      pack_bf16(acc[1][x] * inv, acc[1][2 + x] * inv));
      if (e == 0 && g == 0 && p.lse)
        p.lse[(int64_t)b * p.l_sb + (int64_t)j * p.l_sh] =
            l[x] == 0.f ? -INFINITY : (m[x] + __log2f(l[x])) * 0.6931471805599453f;
    }
  }
};

}  // namespace
}  // namespace hpc
