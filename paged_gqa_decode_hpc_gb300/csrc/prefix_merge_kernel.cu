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
// A CTA has the columns of a (pair, KV head), or a half or quarter of them: thread =
// (column group of 4, row), the 8 rows of a column group adjacent, as the states are
// stored. What bounds it: latency for few pairs, L2 (where the states just written
// still are) for many: 4 KB a state. So which states there are is worked out before
// the wait for the attention kernel (the plan is complete by then: the attention
// kernel lets this one start only after its own wait for it), and 10 states, or 20
// of halves, 30 of quarters, are fetched at once, by bulk copies into shared memory:
// no state waits for another and none takes registers. A long prefix of few
// sequences is cut over many CTAs (8 x 20000 positions: 20 states a pair), which
// whole columns took in rounds: a step of 39.8 us, 37.4 in halves, 35.8 in quarters.
// But CTAs that are not resident when the attention kernel ends have all of this
// ahead of them then (480 pairs and heads, 960 halves: 60.9 -> 63.2 us), so the
// columns are cut as far as all CTAs fit on the GPU at once.
#include <cuda_bf16.h>

#include "hpc_internal.h"
#include "prefix_decode.h"
#include "ptx.cuh"
#include "tc05.cuh"

namespace hpc {

namespace {
constexpr int kListed = 64;  // states listed before the wait
constexpr int kBatch = 10;   // states joined at a time
constexpr uint32_t kRowBytes = 8 * 4;

// kSplit CTAs share the columns of a (pair, KV head).
template <int kSplit>
struct MergeLay {
  static constexpr int kThreads = 256 / kSplit;
  static constexpr int kStates = kBatch * (kSplit < 4 ? kSplit : 3);  // in shared memory
  static_assert(kStates <= 32, "one warp fetches them");
  static constexpr uint32_t kStateBytes = kThreads * 16;
  // CTAs that an SM's 228 KB hold: the states, 8 bytes a listed one, the barrier and 1 KB each
  static constexpr int kResident =
      228 * 1024 / (kStates * (kStateBytes + 2 * kRowBytes) + 8 * kListed + 8 + 1024);
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
constexpr float kLn2 = 0.6931471805599453f;

template <int kSplit>
__global__ void __launch_bounds__(256 / kSplit) prefix_merge_kernel(const PrefixMergeParams p) {
  using Lt = MergeLay<kSplit>;
  constexpr int kThreads = Lt::kThreads, kStates = Lt::kStates;
  constexpr uint32_t kStateBytes = Lt::kStateBytes;
  const int H = p.num_kv_heads, T = p.q_len;
  const int64_t item = blockIdx.x / kSplit;
  const int c0 = (int)(blockIdx.x % kSplit) * (32 / kSplit);  // first column group
  const int pair = (int)(item / H), h = (int)(item % H), b = pair / T, t = pair % T;
  const int row = threadIdx.x & 7, col = threadIdx.x >> 3;
  const int rows_all = p.words[kPxRows], parts = p.words[kPxParts];
  const int2* bounds = reinterpret_cast<const int2*>(p.words + p.bound_off);
  const int4* recs = reinterpret_cast<const int4*>(p.words + p.rec_off);

  // The list of states: for the pair's shared and own work row the first piece's,
  // then those of the parts that continue it.
  __shared__ int64_t s_blk[kListed];
  __shared__ __align__(16) float4 s_o[kStates][kThreads];
  __shared__ __align__(16) float s_m[kStates][8], s_l[kStates][8];
  __shared__ uint64_t s_bar;
  const uint32_t bar = tc05::smem_u32(&s_bar);
  if (threadIdx.x == 0) {
    tc05::mbar_init(bar, 1);
    tc05::fence_barrier_init();
  }
  int64_t home[2] = {-1, -1};
  int lo[2] = {0, 0}, count[2] = {0, 0}, local[2] = {0, t};
  if (rows_all > 0) {
    const int2 s = reinterpret_cast<const int2*>(p.words + p.seq_off)[b];
    const int k = s.x >= 0 ? pair - s.y : 0;
    const int v[2] = {s.x >= 0 ? s.x + k / kPrefixRowPairs : -1, rows_all - p.num_seqs + b};
    int n[2];
    n[0] = s.x >= 0 ? recs[2 * v[0] + 1].x : 0;
    n[1] = recs[2 * v[1] + 1].x;
    local[0] = k % kPrefixRowPairs;
    if (n[0] > 0) home[0] = (int64_t)pair * H + h;
    if (n[1] > 0) home[1] = p.ws.own0 + (int64_t)pair * H + h;
    // parts whose boundary lies inside a row's units (h n, h n + n)
    int hi[2] = {0, 0};
    for (int q0 = 0; q0 < parts; q0 += kThreads) {
      const int q = q0 + threadIdx.x;
      int2 bd = make_int2(INT32_MAX, 0);
      if (q < parts) bd = bounds[q];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        if (n[w] == 0) continue;  // the whole CTA has the same
        const int first = h * n[w];
        lo[w] += __syncthreads_count(bd.x < v[w] || (bd.x == v[w] && bd.y <= first));
        hi[w] += __syncthreads_count(bd.x < v[w] || (bd.x == v[w] && bd.y < first + n[w]));
      }
    }
    for (int w = 0; w < 2; ++w) count[w] = n[w] > 0 ? 1 + hi[w] - lo[w] : 0;
  }
  const int total = count[0] + count[1];
  // state s's block, or -1 (a part without units leaves none)
  auto block_of = [&](int s) -> int64_t {
    const int w = s < count[0] ? 0 : 1, i = w == 0 ? s : s - count[0];
    if (i == 0) return home[w];
    const int q = lo[w] + i - 1;
    const int2 b0 = bounds[q], b1 = bounds[q + 1];
    if (b0.x == b1.x && b0.y == b1.y) return -1;
    return p.ws.cont0 + (int64_t)q * kPrefixRowPairs + local[w];
  };
  for (int s = threadIdx.x; s < total && s < kListed; s += kThreads) s_blk[s] = block_of(s);
  __syncthreads();
  griddep_wait();  // the states
  griddep_launch_dependents();

  float M = -INFINITY, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0, round = 0; s0 < total; s0 += kStates, ++round) {
    const int n = min(kStates, total - s0);
    if (threadIdx.x < 32) {
      const int s = s0 + (int)threadIdx.x;
      int64_t blk = -1;
      if ((int)threadIdx.x < n) blk = s < kListed ? s_blk[s] : block_of(s);
      const int there = __popc(__ballot_sync(0xffffffffu, blk >= 0));
      // the attention kernel's stores before these copies' reads
      asm volatile("fence.proxy.async;" ::: "memory");
      if (threadIdx.x == 0) tc05::mbar_expect_tx(bar, there * (kStateBytes + 2 * kRowBytes));
      __syncwarp();
      if (blk >= 0) {
        bulk_load(tc05::smem_u32(s_m[threadIdx.x]), p.ws.m + blk * 8, kRowBytes, bar);
        bulk_load(tc05::smem_u32(s_l[threadIdx.x]), p.ws.l + blk * 8, kRowBytes, bar);
        bulk_load(tc05::smem_u32(s_o[threadIdx.x]), p.ws.o + blk * 256 + c0 * 8, kStateBytes, bar);
      } else if ((int)threadIdx.x < n) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s_m[threadIdx.x][i] = -INFINITY;
      }
    }
    __syncthreads();
    const unsigned long long t0 = tc05::globaltimer();
    while (!tc05::mbar_try_wait(bar, round & 1)) {
      if (tc05::globaltimer() - t0 > p.timeout_ns) {  // bounded, like every wait of the library
        atomicOr(p.err, HPC_DEVCHK_TIMEOUT);
        break;
      }
    }
    // unrolled over the cells of a batch: absent states and those without a visible
    // key have m = -inf, and what stands in their o is not used
    for (int i0 = 0; i0 < n; i0 += kBatch) {
      float m[kBatch], Mn = M;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        m[i] = i0 + i < n ? s_m[i0 + i][row] : -INFINITY;
        Mn = fmaxf(Mn, m[i]);
      }
      if (Mn == -INFINITY) continue;  // no visible key for this row so far
      const float a = ptx_ex2(M - Mn);
      L *= a;
      acc.x *= a; acc.y *= a; acc.z *= a; acc.w *= a;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float f = ptx_ex2(m[i] - Mn);
        float4 o = s_o[i0 + i][col * 8 + row];
        float l = s_l[i0 + i][row];
        if (m[i] == -INFINITY) {
          o = make_float4(0.f, 0.f, 0.f, 0.f);
          l = 0.f;
        }
        L += l * f;
        acc.x += o.x * f;
        acc.y += o.y * f;
        acc.z += o.z * f;
        acc.w += o.w * f;
      }
      M = Mn;
    }
    __syncthreads();  // the states are used before the next ones arrive
  }
  const float inv = L == 0.f ? 0.f : p.v_scale / L;
  __nv_bfloat16* o = p.out + (int64_t)b * p.o_sb + (int64_t)t * p.o_st +
                     (int64_t)(8 * h + row) * p.o_sh + 4 * (c0 + col);
  const __nv_bfloat162 x = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
  const __nv_bfloat162 y = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&x),
                                            *reinterpret_cast<const uint32_t*>(&y));
  if (p.lse && c0 + col == 0)
    p.lse[(int64_t)b * p.l_sb + (int64_t)t * p.l_st + (int64_t)(8 * h + row) * p.l_sh] =
        L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

template <int kSplit>
cudaError_t launch_split(const PrefixMergeParams& p, int64_t items, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * kSplit));
  cfg.blockDim = dim3(MergeLay<kSplit>::kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix_merge_kernel<kSplit>, p);
}

}  // namespace

cudaError_t launch_prefix_merge(const PrefixMergeParams& p, int num_sms, cudaStream_t stream) {
  const int64_t items = (int64_t)p.num_seqs * p.q_len * p.num_kv_heads;
  if (items * 4 <= (int64_t)num_sms * MergeLay<4>::kResident) return launch_split<4>(p, items, stream);
  if (items * 2 <= (int64_t)num_sms * MergeLay<2>::kResident) return launch_split<2>(p, items, stream);
  return launch_split<1>(p, items, stream);
}

}  // namespace hpc
