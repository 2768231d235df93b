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

}  // namespace

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
