// The pieces of split (sequence, KV head) pairs of a step of several new tokens per
// sequence over a 4-bit cache, joined by log-sum-exp (M = max m_i, l = sum l_i 2^(m_i - M),
// out = sum acc_i 2^(m_i - M) / l) in the owners' order.
//
// A pair's pieces lie with consecutive owners, and an owner begins at most one pair that
// others go on with. Every CTA looks over the owners' records and takes its share of the
// (pair, token) items that there are. A warp is one query head of one of two runs of the
// pieces, a lane four elements, with eight pieces in flight. Latency bounds it: the records, a
// round trip to L2 for every 16 pieces, one exchange in shared memory. (Measured, 13 sequences
// of up to 30011 tokens with 8 drafts each, whole step: 33.1 us with a thread to an element and
// its 8 heads, 31.7 with four runs of four in flight, 29.8 with two of eight, in each of these a
// CTA to an owner and token, most of which have nothing to do; 26.1 with a list of the items.)
#include "hpc_internal.h"
#include "kv4.h"
#include "kv4_state.cuh"
#include "ptx.cuh"

namespace hpc {
namespace {

constexpr int kRuns = 2;

__global__ void __launch_bounds__(kRuns * 256)
    kv4_merge_kernel(const __grid_constant__ Kv4DecodeParams p) {
  __shared__ float4 s_o[kRuns - 1][8][32];
  __shared__ float2 s_ml[kRuns - 1][8];
  __shared__ int4 s_rec[kRuns * 256];
  __shared__ int s_owner[kRuns * 256];
  __shared__ int s_count[kRuns * 8];
  constexpr int kAhead = 8;  // pieces whose loads are in flight
  const int tid = threadIdx.x, lane = tid & 31, g = (tid >> 5) & 7, run = tid >> 8, T = p.q_len;
  griddep_wait();
  griddep_launch_dependents();
  const int n = __ldcg(p.owners);
  for (int base = 0; base < n; base += kRuns * 256) {
    // the owners, of these, that begin such a pair, in their order
    int4 own = make_int4(0, 0, 0, 0);
    if (base + tid < n) own = __ldcg(reinterpret_cast<const int4*>(p.owners + 4 + 4 * (base + tid)));
    const bool begins = own.z > 0;
    const uint32_t mask = __ballot_sync(0xffffffffu, begins);
    if (lane == 0) s_count[tid >> 5] = __popc(mask);
    __syncthreads();
    int before = 0, pairs = 0;
#pragma unroll
    for (int w = 0; w < kRuns * 8; ++w) {
      before += w < (tid >> 5) ? s_count[w] : 0;
      pairs += s_count[w];
    }
    if (begins) {
      const int at = before + __popc(mask & ((1u << lane) - 1u));
      s_owner[at] = base + tid;
      s_rec[at] = own;
    }
    __syncthreads();
    for (int item = blockIdx.x; item < pairs * T; item += gridDim.x) {
      const int ow = s_owner[item / T], t = item % T;
      const int4 rec = s_rec[item / T];
      const int k = rec.z;
      const int lo = (int)((int64_t)k * run / kRuns), hi = (int)((int64_t)k * (run + 1) / kRuns);
      float m = -INFINITY, l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      auto add = [&](float2 ml, float4 y) {
        const float now = fmaxf(m, ml.x);
        const float f = Kv4Slices::factor(m, now), w = Kv4Slices::factor(ml.x, now);
        o = make_float4(o.x * f + y.x * w, o.y * f + y.y * w, o.z * f + y.z * w, o.w * f + y.w * w);
        l = l * f + ml.y * w;
        m = now;
      };
#pragma unroll 1
      for (int i = lo; i < hi; i += kAhead) {
        float4 y[kAhead];
        float2 ml[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          ml[u] = make_float2(-INFINITY, 0.f);
          if (i + u < hi) {
            const int64_t slot = i + u == 0 ? rec.w : 2 * (int64_t)(ow + i + u);
            const int64_t at = (slot * T + t) * 8 + g;
            y[u] = __ldcg(reinterpret_cast<const float4*>(p.ws) + at * 32 + lane);
            ml[u] = __ldcg(p.ws_ml + at);
          }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) add(ml[u], y[u]);
      }
      if (run > 0) {
        s_o[run - 1][g][lane] = o;
        if (lane == 0) s_ml[run - 1][g] = make_float2(m, l);
      }
      __syncthreads();
      if (run == 0) {
#pragma unroll
        for (int r = 0; r < kRuns - 1; ++r) add(s_ml[r][g], s_o[r][g][lane]);
        const int j = rec.y * 8 + g;
        const float f = l == 0.f ? 0.f : p.v_scale / l;
        __nv_bfloat162 x[2] = {__floats2bfloat162_rn(o.x * f, o.y * f),
                               __floats2bfloat162_rn(o.z * f, o.w * f)};
        *reinterpret_cast<uint2*>(p.out + (int64_t)rec.x * p.o_sb + (int64_t)t * p.o_st +
                                  (int64_t)j * p.o_sh + 4 * lane) = *reinterpret_cast<const uint2*>(x);
        if (lane == 0 && p.lse)
          p.lse[(int64_t)rec.x * p.l_sb + (int64_t)t * p.l_st + (int64_t)j * p.l_sh] =
              l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
      }
      __syncthreads();
    }
    __syncthreads();  // (the list is read before the next one is written)
  }
}

}  // namespace

cudaError_t launch_kv4_merge(const Kv4DecodeParams& p, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kRuns * 256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_merge_kernel, p);
}

}  // namespace hpc
