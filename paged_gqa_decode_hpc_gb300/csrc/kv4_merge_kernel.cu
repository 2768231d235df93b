// The pieces of split (sequence, KV head) pairs of a step of several new tokens per
// sequence over a 4-bit cache, joined by log-sum-exp (M = max m_i, l = sum l_i 2^(m_i - M),
// out = sum acc_i 2^(m_i - M) / l) in the owners' order.
//
// A pair's pieces lie with consecutive owners, and an owner begins at most one pair
// that others go on with, so CTA (x, t) takes the pairs begun by owners x, x + grid, ...
// for token t; its warps share the states, which are read once from L2. Latency bounds
// it: the record, the states (9 KB in flight a warp), one exchange in shared memory.
#include "hpc_internal.h"
#include "kv4.h"
#include "kv4_state.cuh"
#include "ptx.cuh"

namespace hpc {
namespace {

constexpr int kWarps = 8;

__global__ void __launch_bounds__(kWarps * 32)
    kv4_merge_kernel(const __grid_constant__ Kv4DecodeParams p) {
  __shared__ float4 s_state[kWarps][9][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.y, T = p.q_len;
  griddep_wait();
  griddep_launch_dependents();
  const int n = __ldcg(p.owners);
  for (int ow = blockIdx.x; ow < n; ow += gridDim.x) {
    const int4 rec = __ldcg(reinterpret_cast<const int4*>(p.owners + 4 + 4 * ow));
    const int k = rec.z;  // pieces; 0: no split pair begins here
    if (k == 0) continue;
    // piece i of the pair: the owner's own slot, then the first slot of the ones behind it
    auto piece = [&](int i) -> const float4* {
      const int64_t slot = i == 0 ? rec.w : 2 * (int64_t)(ow + i);
      return p.ws + (slot * T + t) * kKv4PartFloat4 + lane;
    };
    // warp w takes a run of the pieces, so that the order is the owners'
    const int lo = (int)((int64_t)k * warp / kWarps), hi = (int)((int64_t)k * (warp + 1) / kWarps);
    Kv4State st;
    st.clear();
    for (int i = lo; i < hi; i += 2) st.add2(piece(i), i + 1 < hi ? piece(i + 1) : nullptr);
    if (lo < hi) st.store(&s_state[warp][0][lane]);
    __syncthreads();
    if (warp == 0) {
      st.clear();
      for (int w = 0; w < kWarps; ++w) {
        if ((int64_t)k * w / kWarps == (int64_t)k * (w + 1) / kWarps) continue;
        Kv4State x;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 a = s_state[w][i][lane];
          x.acc[i][0] = a.x; x.acc[i][1] = a.y; x.acc[i][2] = a.z; x.acc[i][3] = a.w;
        }
        const float4 a = s_state[w][8][lane];
        x.m[0] = a.x; x.m[1] = a.y; x.l[0] = a.z; x.l[1] = a.w;
        st.add(x);
      }
      st.write(p, rec.x, t, rec.y, lane);
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_kv4_merge(const Kv4DecodeParams& p, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, p.q_len);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_merge_kernel, p);
}

}  // namespace hpc
