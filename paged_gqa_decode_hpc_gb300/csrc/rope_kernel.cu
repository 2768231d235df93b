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
// What bounds it: HBM, and next to it the instructions that a row costs (8192 tokens
// of 64 + 8 + 8 rows, 336 MB: 52.6 us, 6.38 TB/s; e4m3 cache and queries, half the
// bytes out, 62: the rounding; 64 tokens 3.3 us: latency). Each
// element is read and written once, and a token's 64 (cos, sin) pairs are
// formed once per CTA for all its heads. A CTA is one token; 8 lanes take a
// row, 16 elements each as two 16-byte chunks chosen so that (half layout, R a
// multiple of 16) an element and its partner lie in the same lane: chunk t and
// chunk t + R / 16. Then a pair of pairs turns in four paired-fp32
// instructions, no value moves between lanes, and a lane keeps its cos and sin
// in registers for all rows. (16 lanes a row with the partner fetched by
// shuffles took 83 us for 8192 tokens of 64 + 16 heads.) The rows' loads are in
// flight before the angles are formed. With few tokens the rows of a token are
// spread over several CTAs. Interleaved pairs lie in one lane anyway; in the half
// layout at other R the partners come from a copy of the row in shared memory.
#include <cuda_bf16.h>

#include "cache_ops.h"
#include "convert.cuh"
#include "hpc_internal.h"
#include "ptx.cuh"

namespace hpc {

namespace {

constexpr int kThreads = 128;
constexpr int kLanes = 8;                        // lanes of a row
constexpr int kRowsAtOnce = kThreads / kLanes;
constexpr int kUnroll = 2;                       // rows of a lane loaded together

// kHalfAny: a row's first R elements in shared memory as pairs, its first half once
// more behind them, so that the partners of eight neighbours, elements e + R / 2
// modulo R, are neighbours too. At most 96 words; an odd pitch, so that the four rows
// of a warp lie a bank apart and their lanes' chunks (4 words) in different banks.
constexpr int kRowPitch = 97;

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

// Paired fp32: two lanes' worth of FMA in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// 8 bf16 <-> 4 pairs of floats.
__device__ __forceinline__ void unpack(uint4 u, float2* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 pack(const float2* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[i].x, x[i].y);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint2 quantise(const float2* x, const E4m3Scale& scale) {
  const float v[8] = {x[0].x, x[0].y, x[1].x, x[1].y, x[2].x, x[2].y, x[3].x, x[3].y};
  return quantise_e4m3x8(v, scale);
}
__device__ __forceinline__ float load_weight(const void* w, int32_t dtype, int i) {
  return dtype == HPC_F32 ? ((const float*)w)[i] : __bfloat162float(((const __nv_bfloat16*)w)[i]);
}

// With a norm, or where partners come through shared memory, an element's two
// factors, norm weights included, are read from tables in shared memory for every row
// instead of staying in up to 32 registers, so that 8 CTAs of either fit on an SM
// (8000 tokens of 80 rows: normed, R = 128, 68.8 -> 58.6 us; R = 90 in halves
// 125.6 -> 56.5 us, with the partners as below).
// Element e's place: four neighbours of all chunks, then the other four.
__device__ __forceinline__ int table_at(int e) { return (e & 4) * 16 + (e >> 3) * 4 + (e & 3); }

// CTAs per SM, which bounds the registers (8192 tokens: 52.7 us against 55.6 with 6).
constexpr int kCtas = 8;

template <int LAYOUT, bool NORM>
__global__ void __launch_bounds__(kThreads, kCtas)
    rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr bool kTables = NORM || LAYOUT == kHalfAny;  // see table_at
  __shared__ float s_cos[kHeadDim / 2], s_sin[kHeadDim / 2];
  __shared__ float s_w[NORM ? 2 : 1][kHeadDim];  // norm weights of q and k
  __shared__ uint32_t s_row[LAYOUT == kHalfAny ? kRowsAtOnce : 1][kRowPitch];
  // kTables: what multiplies an element and its partner (cos and signed sin, times
  // the norm weights), of q and of k, by table_at
  __shared__ __align__(16) float s_own[kTables ? 1 + NORM : 1][kHeadDim];
  __shared__ __align__(16) float s_other[kTables ? 1 + NORM : 1][kHeadDim];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t n = blockIdx.x;
  const int tid = threadIdx.x, row_of = tid / kLanes, lane = tid % kLanes;
  const int num_rows = p.num_q_heads + 2 * p.num_kv_heads;
  const int R = p.rot_dim;
  // this lane's two chunks of 8 elements
  int ca = lane, cb = lane + kLanes;
  if (LAYOUT == kHalfLanes) {
    const int hop = R / 16;  // chunks between the halves; chunks past 2 hop pass through
    ca = lane < hop ? lane : 2 * lane;
    cb = lane < hop ? lane + hop : 2 * lane + 1;
  }
  const int ea = 8 * ca, eb = 8 * cb;
  const int pos = p.positions[n], slot = p.slots[n];

  const int step = kRowsAtOnce * gridDim.y;  // rows the token's CTAs take together
  float2 c[kTables ? 1 : 8], s[kTables ? 1 : 8];  // cos, sin of the lane's elements
  int64_t cache_row = 0;
  bool store_kv = false;
  // base: the CTA's first row of a batch of kUnroll rows per lane; all the
  // loop's conditions are the CTA's, so its warps stay whole
  for (int base = kRowsAtOnce * blockIdx.y; base < num_rows; base += step * kUnroll) {
    uint4 raw[kUnroll][2];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = base + row_of + u * step;
      const __nv_bfloat16* src = nullptr;
      if (r < p.num_q_heads)
        src = p.q_in + n * p.qi_sn + r * p.qi_sh;
      else if (r < p.num_q_heads + p.num_kv_heads)
        src = p.k_in + n * p.ki_sn + (r - p.num_q_heads) * p.ki_sh;
      else if (r < num_rows)
        src = p.v_in + n * p.vi_sn + (r - p.num_q_heads - p.num_kv_heads) * p.vi_sh;
      raw[u][0] = src ? *reinterpret_cast<const uint4*>(src + ea) : make_uint4(0u, 0u, 0u, 0u);
      raw[u][1] = src ? *reinterpret_cast<const uint4*>(src + eb) : make_uint4(0u, 0u, 0u, 0u);
    }
    if (base < step) {  // once: this token's angles and place
      if (slot < 0) return;  // padding: nothing is written for it
      if (pos < 0 || pos >= kRopeMaxPosition) {
        if (tid == 0 && blockIdx.y == 0 && p.err) atomicOr(p.err, HPC_DEVCHK_BAD_LENGTH);
        return;
      }
      const int blk = slot / kBlockTokens;
      store_kv = blk < p.num_blocks;
      if (!store_kv && tid == 0 && blockIdx.y == 0 && p.err) atomicOr(p.err, HPC_DEVCHK_BAD_BLOCK);
      cache_row = blk * p.c_sblk + (slot % kBlockTokens) * p.c_sslot;
      if (tid < R / 2) {
        const TurnPair t = turn((float)pos, p.freq_hi[tid], p.freq_lo[tid], p);
        s_cos[tid] = t.c;
        s_sin[tid] = t.s;
      }
      if constexpr (NORM) {
        for (int i = tid; i < 2 * kHeadDim; i += kThreads) {
          const void* w = i < kHeadDim ? p.wq : p.wk;
          s_w[i / kHeadDim][i % kHeadDim] =
              w ? load_weight(w, i < kHeadDim ? p.wq_dtype : p.wk_dtype, i % kHeadDim) : 0.f;
        }
      }
      __syncthreads();
      if constexpr (kTables) {
        static_assert(kThreads == kHeadDim, "an element per thread");
        constexpr bool kPairs = LAYOUT == kInterleaved;
        const int e = tid, r2 = R / 2;
        const int i = e < R ? (kPairs ? e / 2 : (e < r2 ? e : e - r2)) : 0;  // its pair
        const int other = e < R ? (kPairs ? e ^ 1 : (e < r2 ? e + r2 : e - r2)) : e;
        const bool first = kPairs ? (e & 1) == 0 : e < r2;
        for (int kind = 0; kind < 1 + NORM; ++kind) {
          const bool weighted = NORM && (kind == 0 ? p.wq : p.wk) != nullptr;
          const float w = weighted ? s_w[kind][e] : 1.f, wo = weighted ? s_w[kind][other] : 1.f;
          s_own[kind][table_at(e)] = e < R ? s_cos[i] * w : w;
          s_other[kind][table_at(e)] = (first ? -s_sin[i] : s_sin[i]) * wo;
        }
        __syncthreads();
      } else if constexpr (LAYOUT == kHalfLanes) {
        // c, s [0..3]: of the pairs (ea + j, eb + j), j < 8
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = ea + 2 * j < R / 2 ? ea + 2 * j : 0;
          c[j] = make_float2(s_cos[i], s_cos[i + 1]);
          s[j] = make_float2(s_sin[i], s_sin[i + 1]);
        }
      } else {
        // c, s [j]: of the two elements of pair j of the lane's 16; the sine
        // with its sign (new a = a cos - b sin, new b = b cos + a sin)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = (j < 4 ? ea : eb) + 2 * (j & 3), i = e < R ? e / 2 : 0;
          c[j] = make_float2(s_cos[i], s_cos[i]);
          s[j] = make_float2(-s_sin[i], s_sin[i]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (base + u * step >= num_rows) break;
      const int r = base + row_of + u * step;
      const bool is_q = r < p.num_q_heads, is_k = !is_q && r < p.num_q_heads + p.num_kv_heads;
      float2 x[8];
      unpack(raw[u][0], x);
      unpack(raw[u][1], x + 4);
      float2 y[kTables ? 8 : 1];  // the partner of each element
      if constexpr (LAYOUT == kHalfAny) {
        uint32_t* row = s_row[row_of];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t w[4] = {raw[u][q].x, raw[u][q].y, raw[u][q].z, raw[u][q].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int k = (q == 0 ? ea : eb) / 2 + i;
            if (k < R / 2) row[k] = w[i];
            if (2 * k < R / 2) row[R / 2 + k] = w[i];
          }
        }
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          // (past the R elements: whatever is there, not used)
          const int e = (q == 0 ? ea : eb) + R / 2;
          uint32_t w[5];
#pragma unroll
          for (int i = 0; i < 5; ++i) w[i] = row[e / 2 + i];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (e & 1) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
          unpack(make_uint4(w[0], w[1], w[2], w[3]), y + 4 * q);
        }
        __syncwarp();
      }
      float inv = 1.f;
      if constexpr (NORM) {
        float2 q = mul2(x[0], x[0]);
#pragma unroll
        for (int j = 1; j < 8; ++j) q = fma2(x[j], x[j], q);
        float ss = q.x + q.y;
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (is_q ? p.wq != nullptr : (is_k && p.wk != nullptr)) {
          // (rsqrtf is within 2 ulp: 2^-22 next to the result's 2^-8)
          inv = rsqrtf(ss * (1.0f / kHeadDim) + p.eps);
        }
      }
      if constexpr (kTables) {
        if (is_q || is_k) {
          const int kind = NORM && is_k ? 1 : 0;
          if constexpr (LAYOUT != kHalfAny) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              y[j] = LAYOUT == kInterleaved ? make_float2(x[j].y, x[j].x) : x[j ^ 4];
          }
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const int e = (j < 4 ? ea : eb) + 2 * (j & 3);
            const float4 own = *reinterpret_cast<const float4*>(s_own[kind] + table_at(e));
            const float4 oth = *reinterpret_cast<const float4*>(s_other[kind] + table_at(e));
            const float2 none = make_float2(-0.f, -0.f);  // (adding it changes nothing)
            x[j] = fma2(x[j], make_float2(own.x, own.y),
                        e < R ? mul2(y[j], make_float2(oth.x, oth.y)) : none);
            x[j + 1] = fma2(x[j + 1], make_float2(own.z, own.w),
                            e + 2 < R ? mul2(y[j + 1], make_float2(oth.z, oth.w)) : none);
            if constexpr (NORM) {
              x[j] = mul2(x[j], make_float2(inv, inv));
              x[j + 1] = mul2(x[j + 1], make_float2(inv, inv));
            }
          }
        }
      } else if constexpr (LAYOUT == kHalfLanes) {
        if ((is_q || is_k) && ea < R / 2) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 a = x[j], b = x[j + 4], m = mul2(b, s[j]);
            x[j] = fma2(a, c[j], make_float2(-m.x, -m.y));
            x[j + 4] = fma2(b, c[j], mul2(a, s[j]));
          }
        }
      } else if constexpr (LAYOUT == kInterleaved) {
        if (is_q || is_k) {
#pragma unroll
          for (int j = 0; j < 8; ++j)  // R is even: two neighbours turn or stay together
            if ((j < 4 ? ea : eb) + 2 * (j & 3) < R)
              x[j] = fma2(x[j], c[j], mul2(make_float2(x[j].y, x[j].x), s[j]));
        }
      }
      if (is_q) {
        __nv_bfloat16* dst = p.q_out + n * p.qo_sn + r * p.qo_sh;
        *reinterpret_cast<uint4*>(dst + ea) = pack(x);
        *reinterpret_cast<uint4*>(dst + eb) = pack(x + 4);
        if (p.q_fp8) {
          uint8_t* d8 = p.q_fp8 + n * p.qf_sn + r * p.qf_sh;
          *reinterpret_cast<uint2*>(d8 + ea) = quantise(x, p.q_fp8_scale);
          *reinterpret_cast<uint2*>(d8 + eb) = quantise(x + 4, p.q_fp8_scale);
        }
      } else if (r < num_rows && store_kv) {
        const int h = r - p.num_q_heads - (is_k ? 0 : p.num_kv_heads);
        const int64_t off = cache_row + h * p.c_shead;
        if (p.cache_fp8) {
          uint8_t* dst = (uint8_t*)(is_k ? p.k_cache : p.v_cache) + off;
          const E4m3Scale sc = is_k ? p.k_scale : p.v_scale;
          *reinterpret_cast<uint2*>(dst + ea) = quantise(x, sc);
          *reinterpret_cast<uint2*>(dst + eb) = quantise(x + 4, sc);
        } else {
          __nv_bfloat16* dst = (__nv_bfloat16*)(is_k ? p.k_cache : p.v_cache) + off;
          *reinterpret_cast<uint4*>(dst + ea) = is_k ? pack(x) : raw[u][0];
          *reinterpret_cast<uint4*>(dst + eb) = is_k ? pack(x + 4) : raw[u][1];
        }
      }
    }
  }
}

template <bool NORM>
cudaError_t launch_layout(const cudaLaunchConfig_t& cfg, const RopeParams& p, int layout) {
  if (layout == kInterleaved) return cudaLaunchKernelEx(&cfg, rope_kernel<kInterleaved, NORM>, p);
  if (layout == kHalfLanes) return cudaLaunchKernelEx(&cfg, rope_kernel<kHalfLanes, NORM>, p);
  return cudaLaunchKernelEx(&cfg, rope_kernel<kHalfAny, NORM>, p);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int sm_count, cudaStream_t stream) {
  if (p.num_tokens == 0) return cudaSuccess;
  const int rows = p.num_q_heads + 2 * p.num_kv_heads;
  // One CTA per token from four CTAs per SM on; fewer tokens spread their rows. And
  // two per token, if it has rows for them, where one each makes between one and two
  // and a half rounds of resident CTAs: the last round's tail is half as long (1531
  // tokens of 80 rows, e4m3 18.7 -> 16.6, bf16 13.0 -> 11.9 us; 2500: 19.4 -> 18.0,
  // but 608, all resident, 4.9 -> 5.2, and 1531 of 20 rows 5.5 -> 7.4).
  int64_t want = (4LL * sm_count + p.num_tokens - 1) / p.num_tokens;
  const int most = (rows + kRowsAtOnce - 1) / kRowsAtOnce;
  const int layout = p.interleaved ? kInterleaved : p.rot_dim % 16 == 0 ? kHalfLanes : kHalfAny;
  const int64_t resident = (int64_t)sm_count * kCtas;
  if (p.num_tokens > resident && 2 * p.num_tokens <= 5 * resident && most >= 4) want = 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.num_tokens, (unsigned)(want < most ? want : most));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.wq || p.wk ? launch_layout<true>(cfg, p, layout) : launch_layout<false>(cfg, p, layout);
}

}  // namespace hpc
