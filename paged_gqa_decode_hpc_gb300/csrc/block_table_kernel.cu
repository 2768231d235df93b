// Block tables, slot maps and positions of a step, built on the GPU from the
// sequences' lengths, and the way back: the blocks behind a shortened
// sequence returned to the stack of free ones.
//
// With o_b tokens in the cache, n_b new ones and 64-token blocks, sequence b
// takes a_b = ceil((o_b + n_b) / 64) - ceil(o_b / 64) blocks from the top of
// the stack. With A_b and N_b the exclusive prefix sums of a and n,
//   table[b][ceil(o_b / 64) + i] = free[count - 1 - (A_b + i)],   i < a_b
//   token N_b + i of the step: position o_b + i, slot
//   64 * table[b][position / 64] + position % 64,                 i < n_b.
// Every place is a closed form of two prefix sums, so the result is the same
// in every run: no atomic hands out blocks. Truncating pushes the blocks so
// that the first released block ends on top; a truncate to the old lengths
// therefore undoes an append exactly, stack order included.
//
// What bounds it: latency. A decode step of 256 sequences moves 7 KB, and
// prefill chunks of half a million tokens 4 MB. So a call is one launch of
// ONE cluster of 1 or 8 CTAs: every CTA scans all the lengths itself (warp
// shuffles, no exchange between CTAs) and then takes its share of the tokens
// and blocks, finding the sequence of each by binary search in shared memory.
// The lengths and the stack's count may be updated in place: each CTA has read
// them before the cluster barrier, and the first CTA writes them after it; no
// counter in global memory, so nothing is left over between calls and captured
// graphs may run side by side. From kAppendSplitTokens tokens on, 8 SMs are
// too few (index arithmetic: half a million tokens took them 30 us), and the
// tokens go to CTAs on all SMs, the lengths to a second launch behind them.
// (256 sequences, one token each: 5.2 us of the GPU's time; 512 sequences and half a
// million tokens 7.5 us; truncating 1024 sequences 3.6 us.)
//
// A call that cannot be met as a whole (too few free blocks, a table or token
// buffer too small, a bad length) is refused as a whole: every CTA comes to
// the same verdict from the same sums.
#include "cache_ops.h"
#include "hpc_internal.h"
#include "ptx.cuh"

namespace hpc {

namespace {

constexpr int kMaxThreads = 1024;
constexpr int32_t kAppendSplitTokens = 32768;

__device__ __forceinline__ int ceil_block(int x) {
  return (int)(((int64_t)x + kBlockTokens - 1) / kBlockTokens);
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Inclusive block scan of a pair of 64-bit sums (a multiple of 64 threads).
__device__ __forceinline__ void block_scan2(int64_t& a, int64_t& b, int64_t (*warp_tot)[32],
                                            int64_t& tot_a, int64_t& tot_b) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += x;
      b += y;
    }
  }
  if (lane == 31) {
    warp_tot[0][warp] = a;
    warp_tot[1][warp] = b;
  }
  __syncthreads();
  if (warp < 2) {
    int64_t t = lane < (int)(blockDim.x >> 5) ? warp_tot[warp][lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += x;
    }
    warp_tot[warp][lane] = t;
  }
  __syncthreads();
  if (warp > 0) {
    a += warp_tot[0][warp - 1];
    b += warp_tot[1][warp - 1];
  }
  tot_a = warp_tot[0][31];
  tot_b = warp_tot[1][31];
  __syncthreads();  // warp_tot is used again
}

// Last index i of sum[0 .. n] (non-decreasing, sum[0] = 0) with sum[i] <= x;
// for x < sum[n] that is the sequence that holds item x.
__device__ __forceinline__ int find(const int32_t* sum, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sum[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kMaxThreads) append_kernel(const AppendParams p) {
  extern __shared__ int32_t sm[];
  __shared__ int64_t warp_tot[2][32];
  __shared__ int s_bad;  // HPC_DEVCHK_* bits of every thread
  const int B = p.num_seqs, tid = threadIdx.x;
  int32_t* old = sm;            // [B]
  int32_t* tok = sm + B;        // [B + 1] first token of each sequence
  int32_t* blk = tok + B + 1;   // [B + 1] first new block of each sequence
  griddep_wait();
  griddep_launch_dependents();
  const int threads = (int)blockDim.x, rank = (int)blockIdx.x;
  const int gtid = rank * threads + tid, gstep = (int)gridDim.x * threads;

  const int32_t count = *p.count;
  int bad = (count < 0 || count > p.free_cap) ? HPC_DEVCHK_CAPACITY : 0;
  int64_t tokens = 0, blocks = 0;
  if (tid == 0) tok[0] = blk[0] = s_bad = 0;
  __syncthreads();
  for (int base = 0; base < B; base += threads) {
    const int b = base + tid;
    int64_t n = 0, a = 0;
    if (b < B) {
      const int o = p.lens[b], m = p.new_lens[b];
      old[b] = o;
      if (o < 0 || m < 0 || (int64_t)o + m > INT32_MAX) {
        bad |= HPC_DEVCHK_BAD_LENGTH;
      } else {
        const int b1 = ceil_block(o + m);
        if (b1 > p.max_blocks) bad |= HPC_DEVCHK_TABLE_TOO_SHORT;
        n = m;
        a = b1 - ceil_block(o);
      }
    }
    int64_t tn, ta;
    block_scan2(n, a, warp_tot, tn, ta);
    if (b < B) {  // sums past int32 belong to a call that is refused below
      tok[b + 1] = (int32_t)(tokens + n);
      blk[b + 1] = (int32_t)(blocks + a);
    }
    tokens += tn;
    blocks += ta;
  }
  if (tokens > p.cap_tokens) bad |= HPC_DEVCHK_CAPACITY;
  if (blocks > count) bad |= HPC_DEVCHK_NO_BLOCKS;
  if (bad) atomicOr(&s_bad, bad);
  __syncthreads();
  const int any = s_bad;

  if (p.parts == kAppendAll) cluster_sync();  // every CTA has read the lengths and the count
  if (rank == 0 && p.parts != kAppendTokens) {
    if (tid == 0) {
      if (any && p.err) atomicOr(p.err, any);
      *p.count_out = any ? count : (int32_t)(count - blocks);
    }
    for (int b = tid; b < B; b += threads)
      p.lens_out[b] = any ? old[b] : old[b] + (tok[b + 1] - tok[b]);
    for (int b = tid; b <= B; b += threads) p.cu[b] = any ? 0 : tok[b];
  }
  if (p.parts == kAppendLengths) return;
  if (any) {
    for (int64_t t = gtid; t < p.cap_tokens; t += gstep) {
      p.slots[t] = -1;
      p.positions[t] = 0;
    }
    return;
  }
  // an id outside [0, num_blocks) would make slots of another cache's memory
  auto checked = [&](int32_t id) -> int32_t {
    if ((uint32_t)id < (uint32_t)p.num_blocks) return id;
    if (p.err) atomicOr(p.err, HPC_DEVCHK_BAD_BLOCK);
    return -1;
  };
  for (int64_t xi = gtid; xi < blocks; xi += gstep) {
    const int x = (int)xi, b = find(blk, B, x);
    p.table[b * p.bt_sb + ceil_block(old[b]) + (x - blk[b])] = checked(p.free_blocks[count - 1 - x]);
  }
  // four neighbouring tokens per thread: one search, one block id unless they
  // cross into another block or sequence, and 16-byte stores
  for (int64_t g = gtid; 4 * g < p.cap_tokens; g += gstep) {
    const int t0 = (int)(4 * g);
    int32_t slot[4], pos[4];
    int b = t0 < (int)tokens ? find(tok, B, t0) : 0;
    int have = -1, have_b = -1;  // block (of sequence have_b) whose id is in `id`
    int32_t id = -1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int t = t0 + u;
      slot[u] = -1;
      pos[u] = 0;
      if (t < (int)tokens) {
        while (tok[b + 1] <= t) ++b;  // empty sequences hold no token
        pos[u] = old[b] + (t - tok[b]);
        const int j = pos[u] / kBlockTokens;
        if (j != have || b != have_b) {
          const int fresh = j - ceil_block(old[b]);
          id = checked(fresh >= 0 ? p.free_blocks[count - 1 - (blk[b] + fresh)]
                                  : p.table[b * p.bt_sb + j]);
          have = j;
          have_b = b;
        }
        if (id >= 0) slot[u] = id * kBlockTokens + pos[u] % kBlockTokens;
      }
    }
    if (p.vec4 && t0 + 4 <= p.cap_tokens) {
      *reinterpret_cast<int4*>(p.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (t0 + u < p.cap_tokens) {
          p.slots[t0 + u] = slot[u];
          p.positions[t0 + u] = pos[u];
        }
    }
  }
}

__global__ void __launch_bounds__(kMaxThreads) truncate_kernel(const TruncateParams p) {
  extern __shared__ int32_t sm[];
  __shared__ int64_t warp_tot[2][32];
  __shared__ int s_bad;  // HPC_DEVCHK_* bits of every thread
  const int B = p.num_seqs, tid = threadIdx.x;
  int32_t* keep = sm;          // [B]
  int32_t* blk = sm + B;       // [B + 1] first released block of each sequence
  griddep_wait();
  griddep_launch_dependents();
  const int threads = (int)blockDim.x, rank = (int)blockIdx.x;
  const int gtid = rank * threads + tid, gstep = (int)gridDim.x * threads;

  const int32_t count = *p.count;
  int bad = (count < 0 || count > p.free_cap) ? HPC_DEVCHK_CAPACITY : 0;
  int64_t blocks = 0;
  if (tid == 0) blk[0] = s_bad = 0;
  __syncthreads();
  for (int base = 0; base < B; base += threads) {
    const int b = base + tid;
    int64_t a = 0, none = 0;
    if (b < B) {
      const int n = p.lens[b], to = p.to_lens[b];
      const int k = to < n ? to : n;
      keep[b] = k;
      if (n < 0 || to < 0) {
        bad |= HPC_DEVCHK_BAD_LENGTH;
      } else {
        a = ceil_block(n) - ceil_block(k);
        if (a > 0 && ceil_block(n) > p.max_blocks) bad |= HPC_DEVCHK_TABLE_TOO_SHORT;
      }
    }
    int64_t ta, tn;
    block_scan2(a, none, warp_tot, ta, tn);
    if (b < B) blk[b + 1] = (int32_t)(blocks + a);
    blocks += ta;
  }
  if (count + blocks > p.free_cap) bad |= HPC_DEVCHK_CAPACITY;
  if (bad) atomicOr(&s_bad, bad);
  __syncthreads();
  const int any = s_bad;

  if (any && rank == 0)  // refused: the lengths as they were, read again before anyone writes
    for (int b = tid; b < B; b += threads) keep[b] = p.lens[b];
  cluster_sync();  // every CTA has read the lengths and the count
  if (rank == 0) {
    if (tid == 0) {
      if (any && p.err) atomicOr(p.err, any);
      *p.count_out = any ? count : (int32_t)(count + blocks);
    }
    for (int b = tid; b < B; b += threads) p.lens_out[b] = keep[b];
  }
  if (any) return;
  for (int64_t xi = gtid; xi < blocks; xi += gstep) {
    const int x = (int)xi, b = find(blk, B, x);
    int32_t id = p.table[b * p.bt_sb + ceil_block(keep[b]) + (x - blk[b])];
    if ((uint32_t)id >= (uint32_t)p.num_blocks) {
      if (p.err) atomicOr(p.err, HPC_DEVCHK_BAD_BLOCK);
      id = -1;
    }
    p.free_blocks[count + (int)blocks - 1 - x] = id;
  }
}

template <typename P>
cudaError_t launch(void (*kernel)(P), const P& p, int ctas, int threads, bool cluster, size_t smem,
                   std::atomic<uint64_t>& configured, cudaStream_t stream) {
  const cudaError_t e = once_per_device(configured, [&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (3 * kBlockTableMaxSeqs + 2) * (int)sizeof(int32_t));
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Threads of a CTA: 256 where they scan the batch and take its items in one
// go, else 1024 (a small CTA starts and meets its barriers sooner).
int threads_for(int32_t num_seqs, int64_t items) {
  return num_seqs <= 256 && items <= 256 ? 256 : kMaxThreads;
}
// CTAs of the cluster: one while a thread has at most four items, else 8 (the
// portable cluster size).
int cluster_for(int64_t items) { return items <= 4 * kMaxThreads ? 1 : 8; }

}  // namespace

cudaError_t launch_append(const AppendParams& p0, cudaStream_t stream) {
  static std::atomic<uint64_t> configured{0};
  AppendParams p = p0;
  const size_t smem = (size_t)(3 * p.num_seqs + 2) * sizeof(int32_t);
  const int64_t groups = ((int64_t)p.cap_tokens + 3) / 4;
  if (p.cap_tokens <= kAppendSplitTokens) {
    p.parts = kAppendAll;
    return launch(append_kernel, p, cluster_for(groups), threads_for(p.num_seqs, groups), true,
                  smem, configured, stream);
  }
  // prefill chunks: the tokens by as many CTAs as there is work for, then the
  // lengths and the count (perhaps in place) by a second launch
  p.parts = kAppendTokens;
  const int64_t ctas = (groups + kMaxThreads - 1) / kMaxThreads;
  const cudaError_t e = launch(append_kernel, p, (int)(ctas < 304 ? ctas : 304), kMaxThreads, false,
                               smem, configured, stream);
  if (e != cudaSuccess) return e;
  p.parts = kAppendLengths;
  return launch(append_kernel, p, 1, kMaxThreads, true, smem, configured, stream);
}

cudaError_t launch_truncate(const TruncateParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> configured{0};
  const int64_t items = (int64_t)p.num_seqs * p.max_blocks;
  return launch(truncate_kernel, p, cluster_for(items), threads_for(p.num_seqs, items), true,
                (size_t)(2 * p.num_seqs + 1) * sizeof(int32_t), configured, stream);
}

}  // namespace hpc
