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
// row per sequence. A unit is a (KV head, tile) of a work row. Costs are measured
// times (PrefixCosts). A KV head of a row of n tiles costs f + w n. Shared heads
// are long and cut into several pieces, each of which pays the fixed part f (its
// Q, its epilogue) anew, so a tile there costs w X / (X - f), X being the cost of
// a part: P X = S X / (X - f) + O, with S the shared tiles' plain cost and O all
// the rest, is solved by a few steps. Part p of P covers the cost interval
// [p C / P, (p + 1) C / P) of all heads of all rows in order; a boundary inside a
// unit leaves it to the part before, one inside f falls before the head's first
// unit. Parts cost at least kMinPart, or there are fewer of them.
//
// One CTA; what bounds it is latency, 4 to 5 us from its start to its end for 4 to 64
// sequences, code fetched cold included: one trip to memory for all the inputs
// (loaded before anything else), two block-wide scans, binary searches in
// shared memory, 32-bit divisions where the numbers allow. 256 threads for
// small batches (barriers and scans of 8 warps), else 1024.
#include "hpc_internal.h"
#include "prefix_decode.h"
#include "ptx.cuh"

namespace hpc {

namespace {

constexpr int kMaxThreads = 1024;
constexpr int kMinPart = 100;    // 1 us (4 us: 4 x (200 + 1 .. 40) positions 15.7 against 13.0 us)
constexpr int kKeptLens = 1024;  // lengths kept in shared memory

// Inclusive block scan; the total too. One barrier, and one more before the
// totals' cells are used again.
__device__ __forceinline__ int64_t block_scan(int64_t a, int64_t* warp_tot, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, a, o);
    if (lane >= o) a += x;
  }
  if (lane == 31) warp_tot[warp] = a;
  __syncthreads();
  int64_t before = 0, all = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
    const int64_t x = warp_tot[w];
    if (w < warp) before += x;
    all += x;
  }
  *total = all;
  __syncthreads();
  return a + before;
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

// Costs of a KV head of a work row: fixed, and per tile. `stretch`: what a
// piece's fixed part adds to a shared tile, in 64ths.
__device__ __forceinline__ int2 costs(const PrefixCosts& c, bool own, int pairs, int stretch) {
  if (own) return make_int2(c.own_fixed, c.own_tile);
  return make_int2(c.shared_fixed,
                   (pairs > kPrefixTilePairs ? c.two_tile : c.one_tile) * stretch / 64);
}

// a * b / c of non-negative numbers whose result fits 32 bits, c > 0.
__device__ __forceinline__ int64_t muldiv(int64_t a, int b, int c) {
  const int64_t ab = a * b;
  return ab <= UINT32_MAX ? (int64_t)((uint32_t)ab / (uint32_t)c) : a / c * b + a % c * b / c;
}

__global__ void __launch_bounds__(kMaxThreads) prefix_plan_kernel(const PrefixPlanParams p) {
  extern __shared__ int64_t dyn[];
  __shared__ int64_t warp_tot[32];
  __shared__ float2 s_sum[32];
  __shared__ int s_len[kKeptLens];
  __shared__ int s_bad, s_err;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int B = p.num_seqs, G = p.num_groups, T = p.q_len, H = p.num_kv_heads;
  int P = p.num_parts;
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
  // this thread's first inputs, all on their way at once
  const int cu0 = p.cu_groups && tid <= G ? p.cu_groups[tid] : (tid == 0 ? 0 : B);
  const int want0 = tid < G ? p.prefix_lens[tid] : 0;
  const int len0 = tid < B ? p.seq_lens[tid] : 0;
  if (tid == 0) s_bad = s_err = 0;
  for (int g = tid; g <= G; g += nt) {
    cu[g] = g == tid ? cu0 : (p.cu_groups ? p.cu_groups[g] : B);
    gmin[g] = INT32_MAX;
    gcnt[g] = 0;
    gfirst[g] = INT32_MAX;
  }
  __syncthreads();
  for (int g = tid; g <= G; g += nt)
    if (cu[g] < 0 || cu[g] > B || (g == 0 && cu[g] != 0) || (g == G && cu[g] != B) ||
        (g > 0 && cu[g] < cu[g - 1]))
      s_bad = 1;  // every writer stores 1
  __syncthreads();
  if (s_bad) {  // not a partition of the batch: one group without a prefix
    __syncthreads();
    for (int g = tid; g <= G; g += nt) cu[g] = g == 0 ? 0 : B;
    if (tid == 0) s_err = HPC_DEVCHK_BAD_LENGTH;
    __syncthreads();
  }
  auto length = [&](int b) { return b < kKeptLens ? s_len[b] : p.seq_lens[b]; };
  for (int b = tid; b < B; b += nt) {
    const int L = b == tid ? len0 : p.seq_lens[b];
    if (b < kKeptLens) s_len[b] = L;
    if (L < 0) s_err = HPC_DEVCHK_BAD_LENGTH;
    if (L > 0) {
      const int g = find(cu, G, b);
      atomicMin(&gmin[g], L - T + 1);
      atomicAdd(&gcnt[g], 1);
      atomicMin(&gfirst[g], b);
    }
  }
  __syncthreads();
  if (tid < 32) {  // the groups' shared tiles and first work rows, by one warp
    int carry = 0;
    for (int base = 0; base < G; base += 32) {
      const int g = base + tid;
      int s = 0, rows = 0;
      if (g < G) {
        const int want = g == tid ? want0 : p.prefix_lens[g];
        if (want < 0) s_err = HPC_DEVCHK_BAD_LENGTH;
        if (!s_bad && gcnt[g] >= 2) {
          s = min(want, gmin[g]);
          s = min(s > 0 ? s / kBlockTokens : 0, p.max_blocks);
        }
        gtiles[g] = s;
        if (s > 0) rows = ((cu[g + 1] - cu[g]) * T + kPrefixRowPairs - 1) / kPrefixRowPairs;
      }
      int incl = rows;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (tid >= o) incl += x;
      }
      if (g < G) grow[g] = carry + incl - rows;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (tid == 0) grow[G] = carry;
  }
  __syncthreads();
  const int shared = grow[G];
  const int V = shared + B;
  // a shared row's group: groups without rows repeat their neighbour's start,
  // the last one with grow <= v has rows
  auto shared_pairs = [&](int v, int g) {
    return min(kPrefixRowPairs, (cu[g + 1] - cu[g]) * T - kPrefixRowPairs * (v - grow[g]));
  };
  auto record = [&](int v, int4& a, int4& b) {
    if (v < shared) {
      const int g = find(grow, G, v);
      a = make_int4(cu[g] * T + kPrefixRowPairs * (v - grow[g]), shared_pairs(v, g), gfirst[g], 0);
      b = make_int4(gtiles[g], 0, INT32_MAX, 0);
    } else {
      const int s = v - shared, L = max(length(s), 0);
      const int t0 = L > 0 ? gtiles[find(cu, G, s)] : 0;
      a = make_int4(s * T, T, s, t0);
      b = make_int4((int)(((int64_t)L + kBlockTokens - 1) / kBlockTokens) - t0, 1, L, 0);
    }
  };
  int4* recs = reinterpret_cast<int4*>(p.words + p.rec_off);
  // this thread's first row, kept
  int4 mine_a = make_int4(0, 0, 0, 0), mine_b = mine_a;
  if (tid < V) record(tid, mine_a, mine_b);
  // the plain costs of the shared tiles and of all else, and the stretch
  int stretch = 64;
  if (shared > 0) {
    float sum_s = 0.f, sum_o = 0.f;  // estimates: fp32 will do
    for (int v = tid; v < V; v += nt) {
      int4 a = mine_a, b = mine_b;
      if (v != tid) record(v, a, b);
      if (b.x == 0) continue;
      const int2 fw = costs(p.costs, b.y != 0, a.y, 64);
      sum_o += (float)H * (float)fw.x;
      if (b.y) sum_o += (float)H * (float)fw.y * (float)b.x;
      else sum_s += (float)H * (float)fw.y * (float)b.x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sum_s += __shfl_xor_sync(0xffffffffu, sum_s, o);
      sum_o += __shfl_xor_sync(0xffffffffu, sum_o, o);
    }
    if ((tid & 31) == 0) s_sum[tid >> 5] = make_float2(sum_s, sum_o);
    __syncthreads();
    sum_s = sum_o = 0.f;
    for (int w = 0; w < nt / 32; ++w) {  // the same order in every thread
      sum_s += s_sum[w].x;
      sum_o += s_sum[w].y;
    }
    const float F = (float)p.costs.shared_fixed;
    const float per_part = 1.f / (float)P;
    float X = (sum_s + sum_o) * per_part + F, ratio = 1.f;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      ratio = fminf(__fdividef(X, fmaxf(X - F, 1.f)), 4.f);
      X = (sum_s * ratio + sum_o) * per_part;
    }
    stretch = (int)(64.f * ratio);
  }
  int64_t carry = 0;
  for (int base = 0; base < V; base += nt) {
    const int v = base + tid;
    int64_t cost = 0;
    if (v < V) {
      int4 a = mine_a, b = mine_b;
      if (v != tid) record(v, a, b);
      recs[2 * v] = a;
      recs[2 * v + 1] = b;
      if (v >= shared) {  // the sequence's first shared work row, or -1, and its first pair
        const int g = find(cu, G, a.z);
        reinterpret_cast<int2*>(p.words + p.seq_off)[a.z] =
            make_int2(a.w > 0 ? grow[g] : -1, cu[g] * T);
      }
      const int2 fw = costs(p.costs, b.y != 0, a.y, stretch);
      if (b.x > 0) cost = H * (fw.x + (int64_t)fw.y * b.x);
      // the units of a row are counted in 32 bits
      if ((int64_t)H * b.x > INT32_MAX) {
        s_err = HPC_DEVCHK_BAD_LENGTH;
        s_bad = 2;
      }
    }
    int64_t total;
    const int64_t incl = block_scan(cost, warp_tot, &total);
    if (v < V) cum[v] = carry + incl - cost;
    carry += total;
  }
  const int64_t C = carry;
  if (tid == 0) cum[V] = C;
  __syncthreads();
  const bool none = C == 0 || s_bad == 2;
  P = (int)min((int64_t)P, C / kMinPart + 1);
  // boundary q: row v, unit u, and the record of row v for the part behind it
  for (int q = tid; q <= p.num_parts; q += nt) {
    int v = V, u = 0;
    int4 a = make_int4(0, 0, 0, 0), b = a;
    if (q < P && !none) {
      const int64_t c = muldiv(C, q, P);
      v = find(cum, V, c);
      record(v, a, b);
      const int2 fw = costs(p.costs, b.y != 0, a.y, stretch);
      const int64_t head = fw.x + (int64_t)fw.y * b.x, in = c - cum[v];
      const int h = in <= UINT32_MAX && head <= UINT32_MAX ? (int)((uint32_t)in / (uint32_t)head)
                                                           : (int)(in / head);
      const int64_t rest = in - h * head - fw.x;
      u = h * b.x + (rest > 0 ? (int)((uint32_t)(rest + fw.y - 1) / (uint32_t)fw.y) : 0);
    }
    reinterpret_cast<int2*>(p.words + p.bound_off)[q] = make_int2(v, u);
    if (q < p.num_parts) {
      int4* first = reinterpret_cast<int4*>(p.words + p.first_off) + 2 * q;
      first[0] = a;
      first[1] = b;
    }
  }
  if (tid == 0) {
    if (s_err) atomicOr(p.err, s_err);
    p.words[kPxRows] = none ? 0 : V;
    p.words[kPxParts] = none ? 0 : P;
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
  cfg.blockDim = dim3(p.num_seqs <= 256 && p.num_groups < 256 ? 256 : kMaxThreads);
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
