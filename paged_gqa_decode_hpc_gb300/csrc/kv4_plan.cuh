// The plan of a decode step over a 4-bit cache, made by every CTA of a persistent grid from
// the device lengths, and the walk of a CTA's part of it.
//
// A unit is one 64-token tile of one KV head. Units are ordered by sequence, KV head and
// tile, and every (sequence, KV head) pair has PAIR units more ahead of its own, which
// stand for what it costs beside them (its q, its states' way to memory). The units are cut
// into equal parts, one to a CTA; a piece is what of one pair's own units lies in a part.
// (A pool of an eighth of the units in chunks, taken by whoever is done, as the one-token
// step over 8-bit and 16-bit caches has it, cost 3 to 8 us a step here: its pieces are short,
// and a tile is done in a quarter of the time.)
#pragma once
#include <stdint.h>

#include "decode_common.cuh"
#include "hpc_internal.h"
#include "kv4.cuh"
#include "kv4.h"
#include "ptx.cuh"

namespace hpc {
namespace {

constexpr int kWarpPlan = 256;  // sequences that one warp plans by itself
constexpr int kFlagEnd = 1, kFlagWhole = 2;  // of a piece; its pair's number of pieces << 8
// Bookkeeping waits give up this many data waits later: once a data wait has timed out
// every role runs on without copies, and this bookkeeping must then still finish, so that
// the arrival counters return to zero.
constexpr unsigned long long kBookkeepingWaits = 8;

// Whether any of the `threads` threads of barrier `id` says so; they all learn it, and wait for
// each other.
__device__ __forceinline__ bool any_of(int id, int threads, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

// Equal parts [start(o), start(o + 1)) of T units, and the part of a unit. Every unit index
// is below T <= INT32_MAX, so the arithmetic is 32-bit where products fit.
struct PartPlan {
  uint32_t T, P;
  bool small;  // (T + 1) * (P + 1) < 2^32
  __device__ __forceinline__ uint32_t start(uint32_t o) const {
    return small ? o * T / P : (uint32_t)((uint64_t)o * T / P);
  }
  __device__ __forceinline__ uint32_t owner_of(uint32_t x) const {
    return small ? ((x + 1) * P - 1) / T : (uint32_t)(((uint64_t)(x + 1) * P - 1) / T);
  }
};

// Units of a KV head ahead of each sequence, into cu[0 .. B] (cu[0] = 0 is there already);
// *bad where the lengths cannot be. Called by all `threads` (at most 1024) threads of the CTA
// after a barrier. The warp `planner` plans small batches by itself; other warps may look at
// the result only after they have waited for something that it did later.
template <int PAIR>
__device__ __forceinline__ void plan_step(const Kv4DecodeParams& p, int32_t* cu, volatile int* bad,
                                          int32_t* warp_tot, int threads, bool planner) {
  const int B = p.num_seqs, tid = threadIdx.x, lane = tid & 31;
  const uint32_t H = (uint32_t)p.num_kv_heads;
  auto units_of = [&](int32_t len) -> int32_t {  // -1: cannot be
    // more units than INT32_MAX / 1024 are refused, so that no partial sum of a scan pass, of
    // at most 1024 sequences, wraps
    const int64_t n = len > 0 ? ((int64_t)len + kBlockTokens - 1) / kBlockTokens + PAIR : 0;
    return len < 0 || n * H > (int64_t)(INT32_MAX / 1024) ? -1 : (int32_t)n;
  };
  if (B > kWarpPlan) {
    int64_t carry = 0;
    for (int base = 0; base < B; base += threads) {
      const int b = base + tid;
      int32_t n = b < B ? units_of(p.seq_lens[b]) : 0;
      if (n < 0) {
        *bad = 1;
        n = 0;
      }
      int32_t tot;
      const int32_t incl = cta_inclusive_scan(n, warp_tot, &tot);
      if (b < B) cu[b + 1] = (int32_t)(carry + incl);
      carry += tot;
    }
    if (tid == 0 && carry * H > INT32_MAX) *bad = 1;
    __syncthreads();
  } else if (planner) {
    // A lane takes up to 8 neighbouring sequences. (No code for more of them than there are
    // runs: it runs once, and cold.)
    constexpr int kMost = kWarpPlan / 32;
    const int each = (B + 31) >> 5, first = lane * each;
    int32_t n[kMost], sum = 0;
#pragma unroll
    for (int i = 0; i < kMost; ++i) n[i] = i < each && first + i < B ? p.seq_lens[first + i] : 0;
    bool cannot = false;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      if (i >= each) break;
      const int32_t v = units_of(n[i]);
      cannot |= v < 0;
      sum += v < 0 ? 0 : v;
      n[i] = sum;
    }
    int32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      if (i >= each) break;
      if (first + i < B) cu[first + i + 1] = incl - sum + n[i];
    }
    const int64_t carry = __shfl_sync(0xffffffffu, incl, 31);
    cannot = __any_sync(0xffffffffu, cannot) || carry * H > INT32_MAX;
    if (cannot && lane == 0) *bad = 1;
    __syncwarp();
  }
}

// At least MIN units to a CTA.
template <int MIN>
__device__ __forceinline__ PartPlan part_plan(const Kv4DecodeParams& p, const int32_t* cu,
                                              const volatile int* bad) {
  PartPlan M;
  M.T = *bad ? 0u : (uint32_t)cu[p.num_seqs] * (uint32_t)p.num_kv_heads;
  const uint32_t want = (M.T + MIN - 1) / MIN;
  M.P = want < gridDim.x ? want : gridDim.x;
  M.small = (uint64_t)(M.T + 1) * (M.P + 1) < (uint64_t)UINT32_MAX;
  return M;
}

// A pair: sequence, KV head, its first unit and their number (the cost among them).
struct Pair {
  int b;
  uint32_t h, base, nb;
};

// The pair that holds unit x (a warp together).
__device__ __forceinline__ Pair pair_at(const int32_t* cu, int B, uint32_t H, uint32_t x) {
  const int lane = threadIdx.x & 31;
  int at = 0;  // the last b with cu[b] * H <= x: no empty sequence
  for (int n = B; n > 1;) {
    const int step = (n + 31) / 32, i = at + lane * step;
    const uint32_t under =
        __ballot_sync(0xffffffffu, lane * step < n && (uint32_t)cu[i] * H <= x);
    const int k = 31 - __clz((int)under);  // (lane 0's is)
    at += k * step;
    n = n - k * step < step ? n - k * step : step;
  }
  Pair r;
  r.b = at;
  r.base = (uint32_t)cu[at] * H;
  r.nb = (uint32_t)(cu[at + 1] - cu[at]);
  r.h = (x - r.base) / r.nb;
  r.base += r.h * r.nb;
  return r;
}

__device__ __forceinline__ void next_pair(const int32_t* cu, int B, uint32_t H, Pair& r) {
  r.base += r.nb;
  if (++r.h < H) return;
  r.h = 0;
  do ++r.b;
  while (r.b < B && cu[r.b + 1] == cu[r.b]);
  if (r.b < B) r.nb = (uint32_t)(cu[r.b + 1] - cu[r.b]);
}

// A piece: tiles t0 .. t0 + n - 1 of pair (b, h).
struct Piece {
  int b, h, t0, n, flags, slot;
};

// The pieces of part `owner`, in the order in which they are done: the first one, then the
// last where that is the head of a pair that goes on elsewhere, then the whole pairs between
// them. The pieces of split pairs are done early, and their merges overlap the rest.
// ahead(piece) is called before the piece's flags are known, then piece(piece). Returns the
// pair that begins here and goes on: {b, h, pieces, slot}, 0 pieces for none.
template <int PAIR, typename A, typename F>
__device__ __forceinline__ int4 walk_part(const PartPlan& M, const int32_t* cu, int B, uint32_t H,
                                          int owner, A ahead, F piece) {
  int4 begun = make_int4(0, 0, 0, 0);
  const uint32_t lo = M.start(owner), hi = M.start(owner + 1);
  Pair at = pair_at(cu, B, H, lo), second = at;
  uint32_t end = hi;  // of the whole pairs between
  for (int round = 0;; ++round) {
    const uint32_t own = at.base + PAIR, pair_hi = at.base + at.nb;  // the pair's own units
    const uint32_t from = lo > own ? lo : own, to = hi < pair_hi ? hi : pair_hi;
    if (to > from) {  // (else nothing but the pair's cost is here)
      Piece x;
      x.b = at.b;
      x.h = (int)at.h;
      x.t0 = (int)(from - own);
      x.n = (int)(to - from);
      ahead(x);
      const bool whole = from == own && to == pair_hi;
      int k = 1;
      x.slot = -1;
      if (!whole) {
        x.slot = 2 * owner + (own <= lo ? 0 : 1);
        k = (int)(M.owner_of(pair_hi - 1) - M.owner_of(own) + 1);
        if (from == own) begun = make_int4(x.b, x.h, k, x.slot);
      }
      x.flags = (whole ? kFlagWhole : 0) | (k << 8);
      piece(x);
    }
    if (round == 0) {
      if (pair_hi >= hi) break;
      next_pair(cu, B, H, at);
      const Pair tail = pair_at(cu, B, H, hi - 1);
      if (tail.base + tail.nb > hi) {  // it goes on: now, and the pairs before it afterwards
        end = tail.base;
        second = at;
        at = tail;
        continue;
      }
    } else if (round == 1 && end < hi) {
      at = second;
    } else {
      next_pair(cu, B, H, at);
    }
    if (at.base >= end) break;
  }
  return begun;
}

// The copies of a piece's units into a ring of STAGES slots (K then V of a unit), by a whole
// warp: even lanes K, odd lanes V of BATCH units at a time.
template <int STAGES, int BATCH>
struct UnitCopies {
  static_assert(BATCH <= STAGES && BATCH <= 16, "a slot, and two lanes, to each unit of a batch");
  uint32_t ring, full, empty;  // shared memory: slots, their barriers (full: two arrivals)
  uint64_t policy;
  volatile int* abort_flag;
  bool stop;               // a wait gave up, or copies are withheld
  uint32_t g = 0;          // units walked
  uint32_t issued = 0;     // units issued
  uint32_t last_mask = 0;  // where a wait gave up, the lanes that issued behind them
  int raw;                 // this lane's table entry of the piece's first batch, -2: none

  // the entry of unit i0 + lane / 2 of the piece
  __device__ __forceinline__ int entry(const Kv4DecodeParams& p, const Piece& x, int i0) const {
    const int lane = threadIdx.x & 31, i = i0 + (lane >> 1), t = x.t0 + i;
    if (lane >= 2 * BATCH || i >= x.n || t >= p.max_blocks) return -2;
    return __ldg(p.block_table + (int64_t)x.b * p.bt_sb + t);
  }
  __device__ __forceinline__ void ahead(const Kv4DecodeParams& p, const Piece& x) {
    raw = entry(p, x, 0);
  }
  __device__ __forceinline__ void copy(const Kv4DecodeParams& p, const Piece& x) {
    const int lane = threadIdx.x & 31;
    const uint8_t* tiles = (lane & 1 ? p.v : p.k) + (int64_t)x.h * p.c_shead;
    // no more units at once than the ring has slots, so that a unit's slot was last used by
    // one that has been issued already
    for (int i0 = 0; i0 < x.n; i0 += BATCH) {
      const int cnt = x.n - i0 < BATCH ? x.n - i0 : BATCH;
      const bool mine = lane < 2 * cnt;
      const int later = i0 + BATCH < x.n ? entry(p, x, i0 + BATCH) : -2;
      const uint32_t gu = g + (uint32_t)(lane >> 1), slot = gu % STAGES;
      const uint32_t be = empty + 8 * slot, par = ((gu / STAGES) & 1u) ^ 1u, fb = full + 8 * slot;
      const uint32_t dst = ring + slot * (2 * kKv4Tile) + (lane & 1) * kKv4Tile;
      const bool there = raw >= 0 && raw < p.num_blocks;
      if (mine && !there)
        atomicOr(p.err, raw == -2 && x.t0 + i0 + (lane >> 1) >= p.max_blocks
                            ? HPC_DEVCHK_TABLE_TOO_SHORT
                            : HPC_DEVCHK_BAD_BLOCK);
      // (no block: zeros are read in its place)
      const void* src = there ? (const void*)(tiles + (int64_t)raw * p.c_sblk) : kKv4NoTile;
      raw = later;
      g += (uint32_t)cnt;
      if (stop) continue;
      bool todo = mine;
      if (todo) {  // every lane issues as soon as its slot is free
        unsigned long long since = 0;
        for (uint32_t it = 1; todo; ++it) {
          if (mbar_try_wait(be, par)) {
            mbar_arrive_expect_tx(fb, kKv4Tile);
            kv4_copy_tile(dst, src, fb, policy);
            todo = false;
          } else if ((it & 63u) == 0) {
            if (*abort_flag) break;
            if (since == 0) since = globaltimer();
            if (globaltimer() - since > p.timeout_ns) {
              atomicOr(p.err, HPC_DEVCHK_TIMEOUT);
              *abort_flag = 1;
              break;
            }
          }
        }
      }
      __syncwarp();
      last_mask = __ballot_sync(0xffffffffu, mine && !todo);
      stop = __any_sync(0xffffffffu, todo);
      issued = stop ? g - (uint32_t)cnt : g;
    }
  }
  // After an abort: waits (bounded) until the copies in flight have landed.
  __device__ __forceinline__ void drain(const Kv4DecodeParams& p) {
    const int lane = threadIdx.x & 31;
    for (uint32_t u = issued > (uint32_t)STAGES ? issued - STAGES : 0; lane == 0 && u < issued; ++u)
      wait_phase(full + 8 * (u % STAGES), (u / STAGES) & 1u, abort_flag, p.err, 1000000000ull, false);
    // (of a batch that was cut short one tile's copy may be missing: the wait runs out then)
    if (stop && ((last_mask >> lane) & 1u)) {
      const uint32_t u = issued + (uint32_t)(lane >> 1);
      wait_phase(full + 8 * (u % STAGES), (u / STAGES) & 1u, abort_flag, p.err, 1000000000ull, false);
    }
  }
};

}  // namespace
}  // namespace hpc
