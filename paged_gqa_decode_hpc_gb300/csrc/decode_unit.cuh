// The math of one (tile, KV head) unit on one warp, shared by the decode
// kernels: scores S^T = K Q^T of the 8 query heads of a KV head against a
// 64-token tile (mma.sync m16n8k16: M = 16 tokens, N = the 8 heads), the
// online-softmax update and O^T += V^T P^T, on a K/V tile pair that TMA left in
// shared memory with 128-byte swizzle.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace hpc {
namespace {

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                                        uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                                          uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movm_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// lo -> bits 0..15, hi -> bits 16..31
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 bytes (low byte -> low half) to f16x2; exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t x16) {
  uint32_t r;
  const uint16_t h = (uint16_t)(x16 & 0xFFFFu);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
  return r;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(a), "r"(sel));
  return r;
}
// Output coordinate of accumulator element (dm, r): BF16 rows are d = 16dm+g
// (+8); the FP8 V path permutes rows so a thread owns d = 16dm+2g (+1).
template <bool FP8>
__device__ __forceinline__ int acc_d(int dm, int r, int g) {
  return FP8 ? (16 * dm + 2 * g + r) : (16 * dm + g + 8 * r);
}

// Q of one (sequence, kv head) as mma B fragments (B[k = d][n = q head]).
// q0 points at the first query head of the KV head's group, q_sh is the
// stride between query heads (elements).
template <bool FP8>
__device__ __forceinline__ float load_q(const __nv_bfloat16* q0, int64_t q_sh, int lane,
                                        uint32_t (&qf)[8][2]) {
  const int g = lane >> 2, c = lane & 3;
  const __nv_bfloat16* qrow = q0 + (int64_t)g * q_sh;
  if constexpr (!FP8) {
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      qf[ks][0] = __ldg(reinterpret_cast<const uint32_t*>(qrow + 16 * ks + 2 * c));
      qf[ks][1] = __ldg(reinterpret_cast<const uint32_t*>(qrow + 16 * ks + 2 * c + 8));
    }
    return 1.0f;
  } else {
    // Logical k (2c, 2c+1 | 2c+8, 2c+9) of k-step ks maps to d = 16ks + 4c + (0,1 | 2,3),
    // matching the byte order ldmatrix gives the FP8 K tile.
    float v[8][4];
    float amax = 0.f;
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(qrow + 16 * ks + 4 * c));
      v[ks][0] = __uint_as_float(u.x << 16);
      v[ks][1] = __uint_as_float(u.x & 0xFFFF0000u);
      v[ks][2] = __uint_as_float(u.y << 16);
      v[ks][3] = __uint_as_float(u.y & 0xFFFF0000u);
#pragma unroll
      for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fabsf(v[ks][e]));
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    // Power-of-two scale putting max|q| in [2^14, 2^15): f16 holds every
    // bf16 value of that range exactly.
    int e = 0;
    if (amax > 0.f) {
      const int ex = (int)((__float_as_uint(amax) >> 23) & 0xFF) - 127;
      e = 14 - ex;
      e = e < -60 ? -60 : (e > 60 ? 60 : e);
    }
    const float sc = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      qf[ks][0] = pack_f16(v[ks][0] * sc, v[ks][1] * sc);
      qf[ks][1] = pack_f16(v[ks][2] * sc, v[ks][3] * sc);
    }
    return __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e
  }
}

// One (tile, kv head) unit: scores, online softmax update, P.V accumulate.
template <bool FP8>
__device__ __forceinline__ void compute_unit(uint32_t kbase, uint32_t vbase,
                                             const uint32_t (&qf)[8][2], int valid, float sl2,
                                             float (&m)[2], float (&l)[2], float (&acc)[8][4],
                                             int lane) {
  const int r8 = lane & 7;
  const int mi = lane >> 3;
  const int g = lane >> 2;
  float s[4][4];
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) s[mt][0] = s[mt][1] = s[mt][2] = s[mt][3] = 0.f;

  // ---- S^T = K Q^T
  const uint32_t k_lane = kbase + (uint32_t)((r8 + (mi & 1) * 8) * 128);
  if constexpr (!FP8) {
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      const uint32_t off = (uint32_t)((ks >> 2) * 8192 + ((((2 * ks) & 7) + (mi >> 1)) ^ r8) * 16);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        uint32_t a0, a1, a2, a3;
        ldsm_x4(k_lane + mt * 2048 + off, a0, a1, a2, a3);
        mma_bf16(s[mt], a0, a1, a2, a3, qf[ks][0], qf[ks][1]);
      }
    }
  } else {
#pragma unroll
    for (int kp = 0; kp < 4; ++kp) {
      const uint32_t off = (uint32_t)((((2 * kp) + (mi >> 1)) ^ r8) * 16);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        uint32_t r0, r1, r2, r3;
        ldsm_x4(k_lane + mt * 2048 + off, r0, r1, r2, r3);
        mma_f16(s[mt], e4m3x2_to_f16x2(r0), e4m3x2_to_f16x2(r1), e4m3x2_to_f16x2(r0 >> 16),
                e4m3x2_to_f16x2(r1 >> 16), qf[2 * kp][0], qf[2 * kp][1]);
        mma_f16(s[mt], e4m3x2_to_f16x2(r2), e4m3x2_to_f16x2(r3), e4m3x2_to_f16x2(r2 >> 16),
                e4m3x2_to_f16x2(r3 >> 16), qf[2 * kp + 1][0], qf[2 * kp + 1][1]);
      }
    }
  }

  // ---- online softmax (log2 domain); columns 2c (e=0) and 2c+1 (e=1)
  float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int tok = mt * 16 + g + 8 * r;
      float x0 = s[mt][2 * r] * sl2, x1 = s[mt][2 * r + 1] * sl2;
      if (tok >= valid) x0 = x1 = -INFINITY;
      s[mt][2 * r] = x0;
      s[mt][2 * r + 1] = x1;
      mx0 = fmaxf(mx0, x0);
      mx1 = fmaxf(mx1, x1);
    }
  }
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
  }
  const float mn0 = fmaxf(m[0], mx0), mn1 = fmaxf(m[1], mx1);
  const float al0 = ex2(m[0] - mn0), al1 = ex2(m[1] - mn1);
  m[0] = mn0;
  m[1] = mn1;
  float ps0 = 0.f, ps1 = 0.f;
  uint32_t pb[4][2];
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) {
    const float p0 = ex2(s[mt][0] - mn0), p1 = ex2(s[mt][1] - mn1);
    const float p2 = ex2(s[mt][2] - mn0), p3 = ex2(s[mt][3] - mn1);
    ps0 += p0 + p2;
    ps1 += p1 + p3;
    if constexpr (!FP8) {
      pb[mt][0] = movm_trans(pack_bf16(p0, p1));
      pb[mt][1] = movm_trans(pack_bf16(p2, p3));
    } else {
      pb[mt][0] = movm_trans(pack_f16(p0, p1));
      pb[mt][1] = movm_trans(pack_f16(p2, p3));
    }
  }
  l[0] = l[0] * al0 + ps0;
  l[1] = l[1] * al1 + ps1;
#pragma unroll
  for (int dm = 0; dm < 8; ++dm) {
    acc[dm][0] *= al0;
    acc[dm][1] *= al1;
    acc[dm][2] *= al0;
    acc[dm][3] *= al1;
  }

  // ---- O^T += V^T P^T
  if constexpr (!FP8) {
    const uint32_t v_lane = vbase + (uint32_t)(((r8) + ((mi >> 1) << 3)) * 128);
#pragma unroll
    for (int dm = 0; dm < 8; ++dm) {
      const uint32_t off = (uint32_t)((dm >> 2) * 8192 + ((((2 * dm) & 7) + (mi & 1)) ^ r8) * 16);
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) {
        uint32_t a0, a1, a2, a3;
        ldsm_x4_t(v_lane + kt * 2048 + off, a0, a1, a2, a3);
        mma_bf16(acc[dm], a0, a1, a2, a3, pb[kt][0], pb[kt][1]);
      }
    }
  } else {
    const uint32_t v_lane = vbase + (uint32_t)((r8 + ((mi & 1) << 3)) * 128);
#pragma unroll
    for (int dp = 0; dp < 4; ++dp) {
      const uint32_t off = (uint32_t)((((2 * dp) + (mi >> 1)) ^ r8) * 16);
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) {
        uint32_t r0, r1, r2, r3;
        ldsm_x4_t(v_lane + kt * 2048 + off, r0, r1, r2, r3);
        // bytes {0,2} = (token 2c, 2c+1) at even d; bytes {1,3} at odd d
        const uint32_t x0 = prmt(r0, 0x3120), x1 = prmt(r1, 0x3120);
        const uint32_t x2 = prmt(r2, 0x3120), x3 = prmt(r3, 0x3120);
        mma_f16(acc[2 * dp], e4m3x2_to_f16x2(x0), e4m3x2_to_f16x2(x0 >> 16), e4m3x2_to_f16x2(x1),
                e4m3x2_to_f16x2(x1 >> 16), pb[kt][0], pb[kt][1]);
        mma_f16(acc[2 * dp + 1], e4m3x2_to_f16x2(x2), e4m3x2_to_f16x2(x2 >> 16),
                e4m3x2_to_f16x2(x3), e4m3x2_to_f16x2(x3 >> 16), pb[kt][0], pb[kt][1]);
      }
    }
  }
}

}  // namespace
}  // namespace hpc
