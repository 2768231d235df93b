// Joins the partial softmax states of a shared-prefix decode step.
//
// A (pair, KV head) has 8 rows. Its states are the piece that starts its shared
// work row for that head, the parts that continue it, and the same of its own
// work row; in fp32, with M = max m_i:
//   out = v_scale * sum o_i 2^(m_i - M) / sum l_i 2^(m_i - M),
//   lse = ln 2 (M + log2 sum l_i 2^(m_i - M)).
// Which parts continue a piece follows from the plan's boundaries alone, and the
// states are added in that order, so the result does not depend on timing. A
// row that no piece has seen gets out = 0, lse = -inf.
//
// One CTA of 256 threads per (pair, KV head): thread = (column group of 4, row),
// the 8 rows of a column group adjacent, as the states are stored. What bounds
// it: latency for few pairs, HBM (or L2, where the states just written still
// are) for many: 4 KB a state.
#include <cuda_bf16.h>

#include "hpc_internal.h"
#include "prefix_decode.h"
#include "ptx.cuh"

namespace hpc {

namespace {

constexpr int kThreads = 256;
constexpr float kLn2 = 0.6931471805599453f;

__global__ void __launch_bounds__(kThreads) prefix_merge_kernel(const PrefixMergeParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int H = p.num_kv_heads, T = p.q_len;
  const int64_t item = blockIdx.x;
  const int pair = (int)(item / H), h = (int)(item % H), b = pair / T, t = pair % T;
  const int row = threadIdx.x & 7, col = threadIdx.x >> 3;
  const int rows_all = p.words[kPxRows], parts = p.words[kPxParts];
  const int2* bounds = reinterpret_cast<const int2*>(p.words + p.bound_off);
  const int2* seqs = reinterpret_cast<const int2*>(p.words + p.seq_off);
  const int4* recs = reinterpret_cast<const int4*>(p.words + p.rec_off);

  float M = -INFINITY, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](int64_t blk) {
    const float m = p.ws.m[blk * 8 + row], l = p.ws.l[blk * 8 + row];
    const float4 o = p.ws.o[blk * 256 + col * 8 + row];
    if (m == -INFINITY) return;  // the piece held no visible key for this row
    const float Mn = fmaxf(M, m);
    const float a = ptx_ex2(M - Mn), w = ptx_ex2(m - Mn);
    L = L * a + l * w;
    acc.x = acc.x * a + o.x * w;
    acc.y = acc.y * a + o.y * w;
    acc.z = acc.z * a + o.z * w;
    acc.w = acc.w * a + o.w * w;
    M = Mn;
  };
  // the states of work row v for head h; `local`: the pair's number within it
  auto join = [&](int v, int64_t home, int local) {
    const int n = recs[2 * v + 1].x;
    if (n == 0) return;
    const int first = h * n;
    add(home);
    // parts whose boundary lies inside (first, first + n) of row v
    int lo = 0, hi = 0;
    for (int q0 = 0; q0 < parts; q0 += kThreads) {
      const int q = q0 + threadIdx.x;
      int2 bd = make_int2(INT32_MAX, 0);
      if (q < parts) bd = bounds[q];
      lo += __syncthreads_count(bd.x < v || (bd.x == v && bd.y <= first));
      hi += __syncthreads_count(bd.x < v || (bd.x == v && bd.y < first + n));
    }
    for (int q = lo; q < hi; ++q) {
      const int2 b0 = bounds[q], b1 = bounds[q + 1];
      if (b0.x == b1.x && b0.y == b1.y) continue;  // a part without units
      add(p.ws.cont0 + (int64_t)q * kPrefixRowPairs + local);
    }
  };
  if (rows_all > 0) {
    const int2 s = seqs[b];
    if (s.x >= 0) {
      const int k = pair - s.y;
      join(s.x + k / kPrefixRowPairs, (int64_t)pair * H + h, k % kPrefixRowPairs);
    }
    join(rows_all - p.num_seqs + b, p.ws.own0 + (int64_t)pair * H + h, t);
  }
  const float inv = L == 0.f ? 0.f : p.v_scale / L;
  __nv_bfloat16* o = p.out + (int64_t)b * p.o_sb + (int64_t)t * p.o_st +
                     (int64_t)(8 * h + row) * p.o_sh + 4 * col;
  const __nv_bfloat162 x = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
  const __nv_bfloat162 y = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&x),
                                            *reinterpret_cast<const uint32_t*>(&y));
  if (p.lse && col == 0)
    p.lse[(int64_t)b * p.l_sb + (int64_t)t * p.l_st + (int64_t)(8 * h + row) * p.l_sh] =
        L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

}  // namespace

cudaError_t launch_prefix_merge(const PrefixMergeParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.num_seqs * p.q_len * p.num_kv_heads));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix_merge_kernel, p);
}

}  // namespace hpc
