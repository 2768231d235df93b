// Rotary positions of a ragged batch of tokens and the write of their K and V
// rows into the paged cache, in one launch.
//
// For token n at position p, pair i of the first R = rot_dim elements of each
// q and k row (optionally RMS-normalised first) turns by the angle p f_i:
//   (a, b) -> g (a cos - b sin, b cos + a sin),
// with a, b the elements (i, i + R / 2) or, interleaved, (2 i, 2 i + 1), and g
// the table's magnitude; elements past R pass through. Frequencies come ready
// (hpc_rope_init), scaled for long contexts or not, as float pairs.
//
// Angles: p f_i reaches 10^6 radians and more, where fp32 holds it to 0.06.
// It is formed as an unevaluated sum of floats (exact products by FMA), reduced
// by multiples of 2 pi held in three floats, and what the reduction leaves
// below fp32 enters sine and cosine by their derivatives, so cos and sin are
// right to about an ulp for every position below 2^24 (GB300's fp64 rate is
// no way to get there).
//
// What bounds it: HBM. Each element is read and written once, and a token's
// 64 (cos, sin) pairs are formed once per CTA for all its heads: a CTA is one
// token, 16 half-warps take a row each (8 elements, 16 bytes, per lane), so a
// lane keeps its pairs' cos and sin in registers for all rows. All rows' loads
// (5 per half-warp for 64 + 16 heads) are in flight before the angles are
// formed. With few tokens the rows of a token are spread over several CTAs.
// A row's partner elements sit in another lane (half layout, R / 2 a multiple
// of 8: shuffles), in the same lane (interleaved), or anywhere (half layout,
// other R: through shared memory).
#include <cuda_bf16.h>

#include "cache_ops.h"
#include "convert.cuh"
#include "hpc_internal.h"
#include "ptx.cuh"

namespace hpc {

namespace {

constexpr int kThreads = 256;
constexpr int kRowsAtOnce = kThreads / 16;  // one row per half-warp
constexpr int kUnroll = 5;                  // rows of a half-warp loaded together

enum Layout { kInterleaved = 0, kHalfLanes, kHalfAny };

struct TurnPair {
  float c, s;
};

// cos and sin of pos * (f_hi + f_lo), each times `mag`.
__device__ __forceinline__ TurnPair turn(float fpos, float f_hi, float f_lo, const RopeParams& p) {
  const float a = fpos * f_hi;                                    // a + a_lo = pos * f
  const float a_lo = fmaf(fpos, f_lo, fmaf(fpos, f_hi, -a));
  const float k = rintf(a * (1.0f / p.two_pi[0]));
  const float r1 = fmaf(-k, p.two_pi[0], a);                      // exact: multiples of 2^-22 below 4
  const float t = -k * p.two_pi[1], t_lo = fmaf(-k, p.two_pi[1], -t);
  // a_lo reaches half an ulp of a (0.5 at the far end), so it belongs to the
  // argument; only the sums' rounding errors go into the correction
  const float u = t + a_lo, z = u - t, u_err = (t - (u - z)) + (a_lo - z);
  const float r = r1 + u, y = r - r1, r_err = (r1 - (r - y)) + (u - y);
  const float r_lo = r_err + u_err + fmaf(-k, p.two_pi[2], t_lo);
  float s, c;
  sincosf(r, &s, &c);
  return {(c - s * r_lo) * p.magnitude, (s + c * r_lo) * p.magnitude};
}

__device__ __forceinline__ void unpack(uint4 u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint2 quantise(const float (&x)[8], float scale) {
  return make_uint2(quantise_e4m3x4(make_float4(x[0], x[1], x[2], x[3]), scale),
                    quantise_e4m3x4(make_float4(x[4], x[5], x[6], x[7]), scale));
}
// Eight norm weights from element e0 on.
__device__ __forceinline__ void load_weights(const void* w, int32_t dtype, int e0, float (&x)[8]) {
  if (dtype == HPC_F32) {
    const float4 a = *reinterpret_cast<const float4*>((const float*)w + e0);
    const float4 b = *reinterpret_cast<const float4*>((const float*)w + e0 + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    unpack(*reinterpret_cast<const uint4*>((const __nv_bfloat16*)w + e0), x);
  }
}

template <int LAYOUT>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ TurnPair s_turn[kHeadDim / 2];
  __shared__ float s_row[LAYOUT == kHalfAny ? kRowsAtOnce : 1][kHeadDim];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t n = blockIdx.x;
  const int half_warp = threadIdx.x >> 4, chunk = threadIdx.x & 15, e0 = 8 * chunk;
  const int num_rows = p.num_q_heads + 2 * p.num_kv_heads;
  const int pos = p.positions[n], slot = p.slots[n];
  if (slot < 0) return;  // padding: nothing is written for it
  if (pos < 0 || pos >= kRopeMaxPosition) {
    if (threadIdx.x == 0 && blockIdx.y == 0 && p.err) atomicOr(p.err, HPC_DEVCHK_BAD_LENGTH);
    return;
  }
  const int blk = slot / kBlockTokens;
  const bool store_kv = blk < p.num_blocks;
  if (!store_kv && threadIdx.x == 0 && blockIdx.y == 0 && p.err)
    atomicOr(p.err, HPC_DEVCHK_BAD_BLOCK);
  const int64_t cache_row = blk * p.c_sblk + (slot % kBlockTokens) * p.c_sslot + e0;

  const int R = p.rot_dim;
  float c[8], s[8];  // of this lane's elements (interleaved: of its four pairs)
  const int step = kRowsAtOnce * gridDim.y;  // rows the token's CTAs take together
  // base: the CTA's first row of a batch of kUnroll rows per half-warp; all
  // the loop's conditions are the CTA's, so its warps stay whole
  for (int base = kRowsAtOnce * blockIdx.y; base < num_rows; base += step * kUnroll) {
    const int row0 = base + half_warp;
    uint4 raw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = row0 + u * step;
      raw[u] = make_uint4(0u, 0u, 0u, 0u);
      if (r < p.num_q_heads)
        raw[u] = *reinterpret_cast<const uint4*>(p.q_in + n * p.qi_sn + r * p.qi_sh + e0);
      else if (r < p.num_q_heads + p.num_kv_heads)
        raw[u] = *reinterpret_cast<const uint4*>(p.k_in + n * p.ki_sn +
                                                 (r - p.num_q_heads) * p.ki_sh + e0);
      else if (r < num_rows)
        raw[u] = *reinterpret_cast<const uint4*>(
            p.v_in + n * p.vi_sn + (r - p.num_q_heads - p.num_kv_heads) * p.vi_sh + e0);
    }
    if (base < step) {  // once: this token's angles
      if (threadIdx.x < R / 2)
        s_turn[threadIdx.x] = turn((float)pos, p.freq_hi[threadIdx.x], p.freq_lo[threadIdx.x], p);
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // element e0 + j belongs to pair i; past R none is used
        const int e = e0 + j;
        const int i = LAYOUT == kInterleaved ? e / 2 : (e < R / 2 ? e : e - R / 2);
        const TurnPair t = e < R ? s_turn[i] : TurnPair{1.f, 0.f};
        c[j] = t.c;
        // new a = a cos - b sin, new b = b cos + a sin: the sign goes with the element
        const bool lower = LAYOUT == kInterleaved ? (j & 1) == 0 : e < R / 2;
        s[j] = lower ? -t.s : t.s;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = row0 + u * step;
      if (base + u * step >= num_rows) break;
      const bool is_q = r < p.num_q_heads, is_k = !is_q && r < p.num_q_heads + p.num_kv_heads;
      float x[8];
      unpack(raw[u], x);
      const void* w = is_q ? p.wq : p.wk;
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += x[j] * x[j];
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if ((is_q || is_k) && w) {
        float g[8];
        load_weights(w, is_q ? p.wq_dtype : p.wk_dtype, e0, g);
        const float inv = __frcp_rn(__fsqrt_rn(ss * (1.0f / kHeadDim) + p.eps));
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] * inv * g[j];
      }
      // the partner of each element
      float y[8];
      if constexpr (LAYOUT == kInterleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x[j ^ 1];
      } else if constexpr (LAYOUT == kHalfLanes) {
        const int hop = R / 16;  // lanes between the halves
        const int from = chunk < hop ? chunk + hop : (chunk < 2 * hop ? chunk - hop : chunk);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = __shfl_sync(0xffffffffu, x[j], from, 16);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) s_row[half_warp][e0 + j] = x[j];
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = e0 + j;
          y[j] = s_row[half_warp][e < R / 2 ? e + R / 2 : (e < R ? e - R / 2 : e)];
        }
        __syncwarp();
      }
      if (is_q || is_k) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (e0 + j < R) x[j] = fmaf(x[j], c[j], y[j] * s[j]);
      }
      if (is_q) {
        *reinterpret_cast<uint4*>(p.q_out + n * p.qo_sn + r * p.qo_sh + e0) = pack(x);
        if (p.q_fp8)
          *reinterpret_cast<uint2*>(p.q_fp8 + n * p.qf_sn + r * p.qf_sh + e0) =
              quantise(x, p.q_fp8_scale);
      } else if (r < num_rows && store_kv) {
        const int h = r - p.num_q_heads - (is_k ? 0 : p.num_kv_heads);
        void* cache = is_k ? p.k_cache : p.v_cache;
        const int64_t off = cache_row + h * p.c_shead;
        if (p.cache_fp8)
          *reinterpret_cast<uint2*>((uint8_t*)cache + off) =
              quantise(x, is_k ? p.k_scale : p.v_scale);
        else
          *reinterpret_cast<uint4*>((__nv_bfloat16*)cache + off) = is_k ? pack(x) : raw[u];
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int sm_count, cudaStream_t stream) {
  if (p.num_tokens == 0) return cudaSuccess;
  const int rows = p.num_q_heads + 2 * p.num_kv_heads;
  // one CTA per token from two CTAs per SM on; fewer tokens spread their rows
  const int64_t want = (2LL * sm_count + p.num_tokens - 1) / p.num_tokens;
  const int most = (rows + kRowsAtOnce - 1) / kRowsAtOnce;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.num_tokens, (unsigned)(want < most ? want : most));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.interleaved) return cudaLaunchKernelEx(&cfg, rope_kernel<kInterleaved>, p);
  if (p.rot_dim % 16 == 0) return cudaLaunchKernelEx(&cfg, rope_kernel<kHalfLanes>, p);
  return cudaLaunchKernelEx(&cfg, rope_kernel<kHalfAny>, p);
}

}  // namespace hpc
