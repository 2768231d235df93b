// The pieces of split (sequence, KV head) pairs of a step of several new tokens per
// sequence over a 4-bit cache, joined by log-sum-exp (M = max m_i, l = sum l_i 2^(m_i - M),
// out = sum acc_i 2^(m_i - M) / l) in the owners' order.
//
// A pair's pieces lie with consecutive owners, and an owner begins at most one pair that
// others go on with, so CTA (x, t) takes the pairs begun by owners x, x + grid, ... for
// token t. Its 16 warps are four runs of the pieces times the four quarters of a state, each
// with four states in flight. Latency bounds it: the record, a round trip to L2 for every 16
// pieces, one exchange in shared memory.
#include "hpc_internal.h"
#include "kv4.h"
#include "kv4_state.cuh"
#include "ptx.cuh"

namespace hpc {
namespace {

constexpr int kRuns = 4, kThreads = kRuns * 4 * 32;

__global__ void __launch_bounds__(kThreads)
    kv4_merge_kernel(const __grid_constant__ Kv4DecodeParams p) {
  __shared__ float4 s_state[kRuns][4][3][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = warp & 3, run = warp >> 2;
  const int t = blockIdx.y, T = p.q_len;
  griddep_wait();
  griddep_launch_dependents();
  const int n = __ldcg(p.owners);
  for (int ow = blockIdx.x; ow < n; ow += gridDim.x) {
    const int4 rec = __ldcg(reinterpret_cast<const int4*>(p.owners + 4 + 4 * ow));
    const int k = rec.z;  // pieces; 0: no split pair begins here
    if (k == 0) continue;
    // run r takes neighbouring pieces, so that the order is the owners'
    const int lo = (int)((int64_t)k * run / kRuns), hi = (int)((int64_t)k * (run + 1) / kRuns);
    Kv4Slices st;
    st.clear();
    // piece i of the pair: the owner's own slot, then the first slot of the ones behind it
    st.join(hi - lo, e, [&](int i) -> const float4* {
      const int64_t slot = lo + i == 0 ? rec.w : 2 * (int64_t)(ow + lo + i);
      return p.ws + (slot * T + t) * kKv4PartFloat4 + lane;
    });
    float4* mine = s_state[run][e][0] + lane;
    mine[0] = make_float4(st.acc[0][0], st.acc[0][1], st.acc[0][2], st.acc[0][3]);
    mine[32] = make_float4(st.acc[1][0], st.acc[1][1], st.acc[1][2], st.acc[1][3]);
    mine[64] = make_float4(st.m[0], st.m[1], st.l[0], st.l[1]);
    __syncthreads();
    if (run == 0) {
      float4 ml[kRuns - 1], x[kRuns - 1][2];
#pragma unroll
      for (int r = 1; r < kRuns; ++r) {
        const float4* s = s_state[r][e][0] + lane;
        x[r - 1][0] = s[0];
        x[r - 1][1] = s[32];
        ml[r - 1] = s[64];
      }
      st.add(ml, x);
      st.write(p, rec.x, t, rec.y, e, lane);
    }
    __syncthreads();
  }
}

// The same of kv4_tc_kernel's states: accumulators [8 heads][128 elements], maxima and sums
// beside them. A thread is an element; its CTA's four runs of the pieces are joined in shared
// memory.
__global__ void __launch_bounds__(kRuns * 128)
    kv4_tc_merge_kernel(const __grid_constant__ Kv4DecodeParams p) {
  __shared__ float s_o[kRuns - 1][8][128];
  __shared__ float2 s_ml[kRuns - 1][8];
  const int x = threadIdx.x & 127, run = threadIdx.x >> 7, t = blockIdx.y, T = p.q_len;
  griddep_wait();
  griddep_launch_dependents();
  const int n = __ldcg(p.owners);
  for (int ow = blockIdx.x; ow < n; ow += gridDim.x) {
    const int4 rec = __ldcg(reinterpret_cast<const int4*>(p.owners + 4 + 4 * ow));
    const int k = rec.z;
    if (k == 0) continue;
    const int lo = (int)((int64_t)k * run / kRuns), hi = (int)((int64_t)k * (run + 1) / kRuns);
    float m[8], l[8], o[8];
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      m[g] = -INFINITY;
      l[g] = o[g] = 0.f;
    }
    auto add = [&](int g, float2 ml, float y) {
      const float now = fmaxf(m[g], ml.x);
      const float f = Kv4Slices::factor(m[g], now), w = Kv4Slices::factor(ml.x, now);
      o[g] = o[g] * f + y * w;
      l[g] = l[g] * f + ml.y * w;
      m[g] = now;
    };
    for (int i = lo; i < hi; i += 2) {  // two pieces' loads in flight
      float y[2][8];
      float2 ml[2][8];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int64_t slot = i + u == 0 ? rec.w : 2 * (int64_t)(ow + i + u);
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const int64_t at = (slot * T + t) * 8 + g;
          const bool there = i + u < hi;
          y[u][g] = there ? __ldcg(reinterpret_cast<const float*>(p.ws) + at * 128 + x) : 0.f;
          ml[u][g] = there ? __ldcg(p.ws_ml + at) : make_float2(-INFINITY, 0.f);
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int g = 0; g < 8; ++g) add(g, ml[u][g], y[u][g]);
    }
    if (run > 0) {
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        s_o[run - 1][g][x] = o[g];
        if (x == 0) s_ml[run - 1][g] = make_float2(m[g], l[g]);
      }
    }
    __syncthreads();
    if (run == 0) {
#pragma unroll
      for (int r = 0; r < kRuns - 1; ++r)
#pragma unroll
        for (int g = 0; g < 8; ++g) add(g, s_ml[r][g], s_o[r][g][x]);
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        const int j = rec.y * 8 + g;
        p.out[(int64_t)rec.x * p.o_sb + (int64_t)t * p.o_st + (int64_t)j * p.o_sh + x] =
            __float2bfloat16_rn(l[g] == 0.f ? 0.f : o[g] * (p.v_scale / l[g]));
        if (x == 0 && p.lse)
          p.lse[(int64_t)rec.x * p.l_sb + (int64_t)t * p.l_st + (int64_t)j * p.l_sh] =
              l[g] == 0.f ? -INFINITY : (m[g] + __log2f(l[g])) * 0.6931471805599453f;
      }
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_kv4_tc_merge(const Kv4DecodeParams& p, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, p.q_len);
  cfg.blockDim = dim3(kRuns * 128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_tc_merge_kernel, p);
}

cudaError_t launch_kv4_merge(const Kv4DecodeParams& p, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, p.q_len);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_merge_kernel, p);
}

}  // namespace hpc
