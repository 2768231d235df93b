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
// What bounds it: latency for few pairs, L2 (where the states just written still are)
// for many: 4 KB a state. So which states there are is worked out before the wait for
// the attention kernel (the plan is complete by then: the attention kernel lets this
// one start only after its own wait for it; its first word is acquired, so that no line
// of an earlier step's plan in an SM's L1 can stand for it), and the CTAs are cut as small as they
// still all fit on the GPU while that kernel ends; those that do not have all of this
// ahead of them (480 pairs and heads: whole 60.9 us a step, halves 63.2, quarters 66).
// Thread = (column group of 4, row), the 8 rows of a column group adjacent, as the
// states are stored.
//  * Many pairs: a CTA has the columns of a (pair, KV head), or half of them, and
//    fetches 10, or 20, states at once by bulk copies into shared memory: no state
//    waits for another and none takes registers, so that five CTAs fit on an SM.
//  * Few pairs: those are the ones of few heads and long prefixes, cut over many parts
//    (3 sequences on 9000 positions, one KV head: 140 states a pair). A CTA has a half
//    to an eighth of the columns, as many groups of its threads share the states, and
//    their partial joins meet in shared memory. That step takes 19.9 us in eighths,
//    24.5 in quarters, 37.6 with quarters by bulk copies (one warp issuing them), 52
//    with whole columns; 8 sequences on 20000 positions, 8 KV heads, e4m3 (64 pairs and
//    heads, 20 states): 34.8 in quarters, 36.2 by bulk copies, 40.1 whole.
#include <cuda_bf16.h>

#include "hpc_internal.h"
#include "prefix_decode.h"
#include "ptx.cuh"
#include "tc05.cuh"

namespace hpc {

namespace {

constexpr uint32_t kRowBytes = 8 * 4;

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ int32_t ld_acquire(const int32_t* p) {
  int32_t v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
constexpr float kLn2 = 0.6931471805599453f;

// The states of pair `pair` (new token t of sequence b) and KV head h: for the pair's
// shared and own work row the first piece's, then those of the parts that continue it.
struct StateList {
  const PrefixMergeParams& p;
  int64_t home[2] = {-1, -1};
  int lo[2] = {0, 0}, count[2] = {0, 0}, local[2];
  __device__ __forceinline__ StateList(const PrefixMergeParams& params, int pair, int h, int b, int t)
      : p(params), local{0, t} {
    const int H = p.num_kv_heads;
    const int rows_all = ld_acquire(p.words + kPxRows), parts = p.words[kPxParts];
    if (rows_all == 0) return;
    const int2* bounds = reinterpret_cast<const int2*>(p.words + p.bound_off);
    const int4* recs = reinterpret_cast<const int4*>(p.words + p.rec_off);
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
    for (int q0 = 0; q0 < parts; q0 += (int)blockDim.x) {
      const int q = q0 + (int)threadIdx.x;
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
  __device__ __forceinline__ int total() const { return count[0] + count[1]; }
  // state s's block, or -1 (a part without units leaves none)
  __device__ __forceinline__ int64_t block(int s) const {
    const int w = s < count[0] ? 0 : 1, i = w == 0 ? s : s - count[0];
    if (i == 0) return home[w];
    const int q = lo[w] + i - 1;
    const int2* bounds = reinterpret_cast<const int2*>(p.words + p.bound_off);
    const int2 b0 = bounds[q], b1 = bounds[q + 1];
    if (b0.x == b1.x && b0.y == b1.y) return -1;
    return p.ws.cont0 + (int64_t)q * kPrefixRowPairs + local[w];
  }
};

// The joined state of a row (one column group of it) to out and lse.
__device__ __forceinline__ void finish(const PrefixMergeParams& p, int b, int t, int h, int row, int col,
                                       float M, float L, const float4& acc) {
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

// One more state: (M, L, acc) and (m, l, o) joined. A state without a visible key has
// m = -inf, and what stands in its o is not used.
__device__ __forceinline__ void join(float& M, float& L, float4& acc, float m, float l, const float4& o) {
  const float Mn = fmaxf(M, m);
  if (Mn == -INFINITY) return;
  const float a = ptx_ex2(M - Mn), f = ptx_ex2(m - Mn);
  const bool there = m != -INFINITY;
  L = L * a + (there ? l * f : 0.f);
  acc.x = acc.x * a + (there ? o.x * f : 0.f);
  acc.y = acc.y * a + (there ? o.y * f : 0.f);
  acc.z = acc.z * a + (there ? o.z * f : 0.f);
  acc.w = acc.w * a + (there ? o.w * f : 0.f);
  M = Mn;
}

// Many pairs: a CTA each, or two with half of the columns.
constexpr int kBatch = 10;   // states joined at a time
constexpr int kListed = 64;  // states listed before the wait
template <int kSplit>
struct MergeLay {
  static constexpr int kThreads = 256 / kSplit;
  static constexpr int kStates = kBatch * kSplit;  // in shared memory
  static_assert(kStates <= 32, "one warp fetches them");
  static constexpr uint32_t kStateBytes = kThreads * 16;
  // CTAs that an SM's 228 KB hold: the states, 8 bytes a listed one, the barrier and 1 KB each
  static constexpr int resident() {
    return 228 * 1024 / (kStates * (kStateBytes + 2 * kRowBytes) + 8 * kListed + 8 + 1024);
  }
};
template <int kSplit>
__global__ void __launch_bounds__(256 / kSplit)
    prefix_merge_kernel(const __grid_constant__ PrefixMergeParams p) {
  using Lt = MergeLay<kSplit>;
  constexpr int kThreads = Lt::kThreads, kStates = Lt::kStates;
  constexpr uint32_t kStateBytes = Lt::kStateBytes;
  const int H = p.num_kv_heads, T = p.q_len;
  const int64_t item = blockIdx.x / kSplit;
  const int c0 = (int)(blockIdx.x % kSplit) * (32 / kSplit);  // first column group
  const int pair = (int)(item / H), h = (int)(item % H), b = pair / T, t = pair % T;
  const int row = threadIdx.x & 7, col = threadIdx.x >> 3;
  __shared__ int64_t s_blk[kListed];
  __shared__ __align__(16) float4 s_o[kStates][kThreads];
  __shared__ __align__(16) float s_m[kStates][8], s_l[kStates][8];
  __shared__ uint64_t s_bar;
  const uint32_t bar = tc05::smem_u32(&s_bar);
  if (threadIdx.x == 0) {
    tc05::mbar_init(bar, 1);
    tc05::fence_barrier_init();
  }
  const StateList states(p, pair, h, b, t);
  const int total = states.total();
  for (int s = threadIdx.x; s < total && s < kListed; s += kThreads) s_blk[s] = states.block(s);
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
      if ((int)threadIdx.x < n) blk = s < kListed ? s_blk[s] : states.block(s);
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
  finish(p, b, t, h, row, c0 + col, M, L, acc);
}

// Few pairs: kSplit CTAs each, with 1 / kSplit of the columns; kSplit groups of a CTA's
// threads take its states in turn, kFlight of them in flight a thread.
constexpr int kFlight = 8, kFewResident = 3;
constexpr int kListedFew = 320;  // (the parts of 152 SMs twice, and the first pieces)
template <int kSplit>
__global__ void __launch_bounds__(256, kFewResident)
    prefix_merge_few_kernel(const __grid_constant__ PrefixMergeParams p) {
  constexpr int kThreads = 256;
  constexpr int kLanes = kThreads / kSplit;
  const int H = p.num_kv_heads, T = p.q_len;
  const int64_t item = blockIdx.x / kSplit;
  const int pair = (int)(item / H), h = (int)(item % H), b = pair / T, t = pair % T;
  const int group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes, row = lane & 7;
  const int col = (int)(blockIdx.x % kSplit) * (32 / kSplit) + (lane >> 3);
  __shared__ int64_t s_blk[kListedFew];
  __shared__ float4 s_acc[kThreads];
  __shared__ float s_M[kThreads], s_L[kThreads];
  const StateList states(p, pair, h, b, t);
  const int total = states.total();
  for (int s = threadIdx.x; s < total && s < kListedFew; s += kThreads) s_blk[s] = states.block(s);
  __syncthreads();
  griddep_wait();  // the states
  griddep_launch_dependents();
  float M = -INFINITY, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = group; s0 < total; s0 += kSplit * kFlight) {
    float m[kFlight], l[kFlight];
    float4 o[kFlight];
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const int s = s0 + kSplit * i;
      const int64_t blk = s < total ? (s < kListedFew ? s_blk[s] : states.block(s)) : -1;
      m[i] = -INFINITY;
      l[i] = 0.f;
      o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (blk >= 0) {
        m[i] = __ldcg(p.ws.m + blk * 8 + row);
        l[i] = __ldcg(p.ws.l + blk * 8 + row);
        o[i] = __ldcg(p.ws.o + blk * 256 + col * 8 + row);
      }
    }
    float Mn = M;
#pragma unroll
    for (int i = 0; i < kFlight; ++i) Mn = fmaxf(Mn, m[i]);
    if (Mn == -INFINITY) continue;  // no visible key for this row so far
    const float a = ptx_ex2(M - Mn);
    L *= a;
    acc.x *= a; acc.y *= a; acc.z *= a; acc.w *= a;
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      if (m[i] == -INFINITY) continue;
      const float f = ptx_ex2(m[i] - Mn);
      L += l[i] * f;
      acc.x += o[i].x * f;
      acc.y += o[i].y * f;
      acc.z += o[i].z * f;
      acc.w += o[i].w * f;
    }
    M = Mn;
  }
  s_M[threadIdx.x] = M;
  s_L[threadIdx.x] = L;
  s_acc[threadIdx.x] = acc;
  __syncthreads();
  if (group != 0) return;
#pragma unroll
  for (int g = 1; g < kSplit; ++g)
    join(M, L, acc, s_M[g * kLanes + lane], s_L[g * kLanes + lane], s_acc[g * kLanes + lane]);
  finish(p, b, t, h, row, col, M, L, acc);
}

template <typename K>
cudaError_t launch(K kernel, int64_t ctas, int threads, const PrefixMergeParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_prefix_merge(const PrefixMergeParams& p, int num_sms, cudaStream_t stream) {
  const int64_t items = (int64_t)p.num_seqs * p.q_len * p.num_kv_heads, sms = num_sms;
  if (items * 8 <= sms * kFewResident) return launch(prefix_merge_few_kernel<8>, items * 8, 256, p, stream);
  if (items * 4 <= sms * kFewResident) return launch(prefix_merge_few_kernel<4>, items * 4, 256, p, stream);
  if (items <= sms) return launch(prefix_merge_few_kernel<2>, items * 2, 256, p, stream);
  if (items * 2 <= sms * MergeLay<2>::resident())
    return launch(prefix_merge_kernel<2>, items * 2, MergeLay<2>::kThreads, p, stream);
  return launch(prefix_merge_kernel<1>, items, MergeLay<1>::kThreads, p, stream);
}

}  // namespace hpc
