// The work list of a shared-prefix decode step, from device lengths.
//
// Group g (sequences cu_groups[g] .. cu_groups[g+1] - 1) shares its first
// prefix_lens[g] positions. Its shared tiles are the whole 64-token blocks
// among them that every new token of every non-empty sequence of the group
// sees; at least two such sequences, or nothing is shared:
//   s_g = floor(min(prefix_lens[g], min_b (L_b - q_len + 1)) / 64).
// So no shared tile needs a mask, and what lies behind is the sequences' own:
// sequence b has ceil(L_b / 64) - s_g tiles of its own.
// Work rows: for every group with s_g > 0, its pairs in sets of 32; then one
// row per sequence. A unit is a (KV head, tile) of a work row. A KV head of a
// row of n tiles costs f + w n, f and w by the row's kind (measured times, see
// PrefixCosts), and part p of P covers the cost interval [p C / P, (p + 1) C / P)
// of all heads of all rows in order; a boundary inside a unit leaves it to the
// part before, one inside f falls before the head's first unit.
//
// One CTA of 1024 threads; what bounds it is latency (a few block-wide scans).
#include "hpc_internal.h"
#include "prefix_decode.h"
#include "ptx.cuh"

namespace hpc {

namespace {

constexpr int kThreads = 1024;

__device__ __forceinline__ int64_t block_scan(int64_t a, int64_t* warp_tot, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, a, o);
    if (lane >= o) a += x;
  }
  if (lane == 31) warp_tot[warp] = a;
  __syncthreads();
  if (warp == 0) {
    int64_t t = warp_tot[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += x;
    }
    warp_tot[lane] = t;
  }
  __syncthreads();
  if (warp > 0) a += warp_tot[warp - 1];
  *total = warp_tot[31];
  __syncthreads();
  return a;
}

// Last i in [0, n) with a[i] <= x (a non-decreasing, a[0] <= x).
template <typename T>
__device__ __forceinline__ int find(const T* a, int n, T x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Costs of a KV head of a work row: fixed, and per tile.
__device__ __forceinline__ int2 costs(const PrefixCosts& c, bool own, int pairs) {
  if (own) return make_int2(c.own_fixed, c.own_tile);
  return make_int2(c.shared_fixed, pairs > kPrefixTilePairs ? c.two_tile : c.one_tile);
}

__global__ void __launch_bounds__(kThreads) prefix_plan_kernel(const PrefixPlanParams p) {
  extern __shared__ int64_t dyn[];
  __shared__ int64_t warp_tot[32];
  __shared__ int s_bad, s_err;
  const int tid = threadIdx.x, B = p.num_seqs, G = p.num_groups, T = p.q_len, H = p.num_kv_heads;
  // [G + 1] each: group starts, least visible length, non-empty sequences, first of them,
  // shared tiles, first work row
  int32_t* cu = reinterpret_cast<int32_t*>(dyn);
  int32_t* gmin = cu + G + 1;
  int32_t* gcnt = gmin + G + 1;
  int32_t* gfirst = gcnt + G + 1;
  int32_t* gtiles = gfirst + G + 1;
  int32_t* grow = gtiles + G + 1;
  int64_t* cum = dyn + (6LL * (G + 1) + 1) / 2;  // [rows + 1] cost before each work row
  griddep_wait();
  griddep_launch_dependents();
  if (tid == 0) s_bad = s_err = 0;
  __syncthreads();
  for (int g = tid; g <= G; g += kThreads) {
    cu[g] = p.cu_groups ? p.cu_groups[g] : (g == 0 ? 0 : B);
    gmin[g] = INT32_MAX;
    gcnt[g] = 0;
    gfirst[g] = INT32_MAX;
  }
  __syncthreads();
  for (int g = tid; g <= G; g += kThreads)
    if (cu[g] < 0 || cu[g] > B || (g == 0 && cu[g] != 0) || (g == G && cu[g] != B) ||
        (g > 0 && cu[g] < cu[g - 1]))
      s_bad = 1;  // every writer stores 1
  __syncthreads();
  if (s_bad) {  // not a partition of the batch: one group without a prefix
    __syncthreads();
    for (int g = tid; g <= G; g += kThreads) cu[g] = g == 0 ? 0 : B;
    if (tid == 0) s_err = HPC_DEVCHK_BAD_LENGTH;
    __syncthreads();
  }
  for (int b = tid; b < B; b += kThreads) {
    const int L = p.seq_lens[b];
    if (L < 0) s_err = HPC_DEVCHK_BAD_LENGTH;
    if (L > 0) {
      const int g = find(cu, G, b);
      atomicMin(&gmin[g], L - T + 1);
      atomicAdd(&gcnt[g], 1);
      atomicMin(&gfirst[g], b);
    }
  }
  __syncthreads();
  int64_t carry = 0;
  for (int base = 0; base < G; base += kThreads) {
    const int g = base + tid;
    int64_t rows = 0;
    if (g < G) {
      const int want = p.prefix_lens[g];
      if (want < 0) s_err = HPC_DEVCHK_BAD_LENGTH;
      int s = 0;
      if (!s_bad && gcnt[g] >= 2) {
        s = min(want, gmin[g]);
        s = min(s > 0 ? s / kBlockTokens : 0, p.max_blocks);
      }
      gtiles[g] = s;
      if (s > 0)
        rows = ((int64_t)(cu[g + 1] - cu[g]) * T + kPrefixRowPairs - 1) / kPrefixRowPairs;
    }
    int64_t total;
    const int64_t incl = block_scan(rows, warp_tot, &total);
    if (g < G) grow[g] = (int32_t)(carry + incl - rows);
    carry += total;
  }
  const int shared = (int)carry;
  const int V = shared + B;
  if (tid == 0) grow[G] = shared;
  __syncthreads();
  int64_t units = 0;  // of this thread's rows
  PrefixRec* recs = reinterpret_cast<PrefixRec*>(p.words + p.rec_off);
  carry = 0;
  for (int base = 0; base < V; base += kThreads) {
    const int v = base + tid;
    int64_t cost = 0;
    if (v < V) {
      PrefixRec r;
      r.pad = 0;
      if (v < shared) {
        // groups without rows repeat their neighbour's start: the last one with
        // grow <= v has rows
        const int g = find(grow, G, v);
        const int k = v - grow[g], all = (cu[g + 1] - cu[g]) * T;
        r.pair0 = cu[g] * T + kPrefixRowPairs * k;
        r.pairs = min(kPrefixRowPairs, all - kPrefixRowPairs * k);
        r.table = gfirst[g];
        r.tile0 = 0;
        r.tiles = gtiles[g];
        r.own = 0;
        r.len = INT32_MAX;
      } else {
        const int b = v - shared, L = max(p.seq_lens[b], 0), g = find(cu, G, b);
        const int t0 = L > 0 ? gtiles[g] : 0;
        r.pair0 = b * T;
        r.pairs = T;
        r.table = b;
        r.tile0 = t0;
        r.tiles = (int)(((int64_t)L + kBlockTokens - 1) / kBlockTokens) - t0;
        r.own = 1;
        r.len = L;
        int32_t* sr = p.words + p.seq_off + 2 * b;
        // the sequence's first shared work row and pair, or -1
        const bool has = t0 > 0;
        sr[0] = has ? grow[g] : -1;
        sr[1] = cu[g] * T;
      }
      const int2 fw = costs(p.costs, r.own != 0, r.pairs);
      if (r.tiles > 0) cost = H * (fw.x + (int64_t)fw.y * r.tiles);
      units += (int64_t)H * r.tiles;
      int4* dst = reinterpret_cast<int4*>(recs + v);
      const int4* src = reinterpret_cast<const int4*>(&r);
      dst[0] = src[0];
      dst[1] = src[1];
    }
    int64_t total;
    const int64_t incl = block_scan(cost, warp_tot, &total);
    if (v < V) cum[v] = carry + incl - cost;
    carry += total;
  }
  const int64_t C = carry;
  int64_t all_units;
  block_scan(units, warp_tot, &all_units);
  if (tid == 0) cum[V] = C;
  __syncthreads();
  // units of a work row are counted in 32 bits by its readers
  const bool huge = all_units > INT32_MAX;
  const int P = huge ? 0 : (int)min((int64_t)p.num_parts, all_units);
  for (int q = tid; q <= P; q += kThreads) {
    int v = V, u = 0;
    if (q < P) {
      const int64_t c = C / P * q + C % P * q / P;
      v = find(cum, V, c);
      const PrefixRec r = recs[v];  // written by this CTA before the barrier
      const int2 fw = costs(p.costs, v >= shared, r.pairs);
      const int64_t head = fw.x + (int64_t)fw.y * r.tiles, in = c - cum[v];
      const int h = (int)(in / head);
      const int64_t rest = in - h * head - fw.x;
      u = h * r.tiles + (rest > 0 ? (int)((rest + fw.y - 1) / fw.y) : 0);
    }
    p.words[p.bound_off + 2 * q] = v;
    p.words[p.bound_off + 2 * q + 1] = u;
  }
  if (tid == 0) {
    if (huge) s_err = HPC_DEVCHK_BAD_LENGTH;
    if (s_err) atomicOr(p.err, s_err);
    p.words[kPxRows] = huge ? 0 : V;
    p.words[kPxShared] = shared;
    p.words[kPxParts] = P;
  }
}

}  // namespace

cudaError_t launch_prefix_plan(const PrefixPlanParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = once_per_device(configured, [] {
    return cudaFuncSetAttribute(prefix_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                200 * 1024);
  });
  if (e != cudaSuccess) return e;
  const int64_t rows = 2LL * p.num_seqs + (int64_t)p.num_seqs * p.q_len / kPrefixRowPairs + 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes =
      (size_t)(((6LL * (p.num_groups + 1) + 1) / 2 + rows + 1) * sizeof(int64_t));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix_plan_kernel, p);
}

}  // namespace hpc
