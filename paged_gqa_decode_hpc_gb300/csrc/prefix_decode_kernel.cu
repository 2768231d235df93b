// Shared-prefix split-KV decode attention on the 5th-generation tensor cores
// (tcgen05), for sm_103a.
//
// Sequences of a group share their first blocks (a system prompt, a document).
// For one KV head the q_len x 8 query rows of all of them attend to the same K
// and V there, so the shared tiles are a dense contraction over up to 256 rows
// per CTA and are read once for all, not once per sequence; each sequence's own
// tiles follow. Both kinds of work are the same loop over (work row, KV head,
// tiles) pieces of one plan (prefix_plan_kernel.cu), cut into parts of equal
// cost, one persistent CTA per part: compute-bound shared pieces and
// HBM-bound own pieces run side by side on different SMs. Every piece leaves
// partial softmax states (m, l, o), in fp32, that the merge kernel joins:
//   out = sum o_i 2^(m_i - M) / sum l_i 2^(m_i - M),  M = max m_i.
//
// The CTA has two pipelines g = 0, 1, each with its own S, P and O in tensor
// memory, a softmax warpgroup (thread = query row = TMEM lane) and an MMA warp;
// one TMA producer warp feeds both from one K / V ring (for e4m3 caches 4
// converter warps widen an e4m3 ring into it). A piece runs in one of two ways:
//  * two row tiles (more than 16 pairs): pipeline g holds rows 128 g ..
//    128 g + 127 (16 pairs x 8 heads) and works on every tile;
//  * one row tile: both hold the same rows, pipeline g takes the tiles of
//    parity g, and at the end of the piece warpgroup 0 joins the two states.
//    A lone chain S -> softmax -> P V leaves the tensor cores and the ring
//    idle between its steps; two chains on alternate tiles fill in for each
//    other.
// Own pieces of a single new token have 8 rows only, and a chain through tensor
// memory costs each tile its full latency (as own pieces of several tokens do: about
// 0.6 us a tile and 3 us a piece). They run as warp pieces, 0.55 us a tile and 0.3 a
// piece (e4m3 0.32 and 0.7): the 8 softmax warps take tiles in
// turn, each alone from the ring with mma.sync (8 heads = the N of one
// instruction; decode_unit.cuh) and fp32 state in registers; e4m3 tiles are read
// as they are. At the end each warp leaves its state in shared memory (the Q
// slots, which own pieces do not need and which follow all shared ones) and goes
// on; the MMA warps join the 8 states of alternate pieces and write them out.
// Q sits in two slots of 128 rows: one per row tile, or, with one row tile,
// used in turn, so that the next piece's Q loads early.
//
// The tile loop is the extend kernel's: S_j = Q K_j^T (M 128, N 64, K 128);
// online softmax in the log2 domain, the running maximum moved only when it
// grows by more than 8; P as 16-bit pairs back to tensor memory (bf16 for a
// bf16 cache, whose V has bf16's range: 2^-8 of each probability; f16 for e4m3:
// 2^-11, see below, and at least 2^-25 of the row's largest); O += P V_j (M 128, N 128, K 64). Row sums are fp32 of the
// unrounded probabilities.
// E4m3 caches run the MMAs in fp16: every e4m3 value is an f16 value, and each
// query row is converted in place with a power-of-two scale putting its largest
// |q| in [2^14, 2^15), and the sign of the K scale.
// Slots of a sequence's last block behind its end may hold anything (NaN in V
// would pass 0 * NaN into O): their scores are masked, and their V rows are
// zeroed in shared memory before the P V product reads them.
// Every wait is bounded; a timeout sets the error bit, all roles stop issuing,
// and the CTA drains its copies and MMAs and frees its tensor memory.
//
// What bounds it (64 sequences of 32768 shared and 128 .. 2048 own positions, 8 KV
// heads, bf16: 83 us of a step of 90, 431 MB from memory): a shared tile of two row
// tiles takes 0.82 us, of which the tensor pipe works 0.7 (S with N = 64 reads Q from
// shared memory again for every tile: 384 of its cycles where the MMAs need 269) and
// the softmax 0.6; own tiles take what their loads take, and more loads in flight do
// not help: five loading threads instead of one (92.8 -> 98.7 us) and tiles asked into
// L2 ten ahead of the ring (90.4 -> 98.9 us) were both slower.
#include <cfloat>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "decode_unit.cuh"
#include "hpc_decode.h"
#include "hpc_internal.h"
#include "prefix_decode.h"
#include "ptx.cuh"
#include "tc05.cuh"

namespace hpc {

namespace {

using namespace tc05;

constexpr int kRows = 128;                          // rows of one MMA tile
constexpr int kGroupRows = 8;                       // query heads per KV head
constexpr uint32_t kQSlotBytes = kRows * 128 * 2;   // 32 KB: two 16 KB column halves
constexpr uint32_t kQHalfBytes = kQSlotBytes / 2;
constexpr uint32_t kKVTileBytes = 64 * 128 * 2;     // 16 KB: two 8 KB column halves
constexpr uint32_t kStageBytes = 2 * kKVTileBytes;  // K + V
constexpr uint32_t kKVTileBytes8 = 64 * 128;        // 8 KB: one e4m3 K or V tile
constexpr uint32_t kStageBytes8 = 2 * kKVTileBytes8;
// tensor memory of a pipeline: two S buffers of 64 columns (P of a tile overwrites
// the first half of its S), O
constexpr uint32_t kColS = 0, kColO = 128, kColsPerPipe = 256;
constexpr float kRescaleThreshold = 8.0f;           // log2 units

template <bool FP8>
struct Lay {
  static constexpr int kConvWarps = FP8 ? 4 : 0;
  static constexpr int kConvWarp0 = 8;
  static constexpr int kProducerWarp = 8 + kConvWarps, kMmaWarp0 = kProducerWarp + 1;
  // whole warpgroups (one warp idle), so that registers can move to the softmax ones
  static constexpr int kThreads = FP8 ? 512 : 384;
  // K + V rings, 16-bit and e4m3. Of the e4m3 cache's 160 KB more slots went to the
  // ring that copies land in: with 4 + 2, loads beside own pieces that saturate the
  // memory came late (6 groups of 4 to 20, 1300 .. 14300 shared: 65.1 against 62.3 us).
  static constexpr int kStages = FP8 ? 3 : 5;
  static constexpr int kStages8 = FP8 ? 4 : 0;
  // warp pieces: the 16-bit ring, or, all as e4m3 slots, the space of both rings
  static constexpr int kWStages = FP8 ? 2 * kStages + kStages8 : kStages;
  static constexpr uint32_t kWStageBytes = FP8 ? kStageBytes8 : kStageBytes;
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffKV = 2 * kQSlotBytes;
  static constexpr uint32_t kOffKV8 = kOffKV + kStages * kStageBytes;
  static constexpr uint32_t kOffBar = kOffKV8 + kStages8 * kStageBytes8;
  // q_full[2], q_empty[2], q_ready[2], kv_full[S], kv_empty[S], kv8_full[S8],
  // kv8_empty[S8], x_full, x_free, dep_full[2], dep_free[2], q_done, per pipeline:
  // s_full[2], p_full[2], pv_done[2], drain; FP8: w_full[W], w_empty[W]
  static constexpr int kNumBars =
      6 + 2 * kStages + 2 * kStages8 + 7 + 14 + (FP8 ? 2 * kWStages : 0);
  // int8 [2 slots][2 fills][128]: a warpgroup that lags may still read the scales
  // of a slot's fill while the next one is converted, never the one after that
  static constexpr uint32_t kOffScale = kOffBar + 8 * kNumBars;
  static constexpr uint32_t kOffX = kOffScale + (FP8 ? 4 * kRows : 0);  // float [2][128]
  static constexpr uint32_t kOffWord = kOffX + 2 * kRows * 4;  // warp pieces: tile in each slot
  static constexpr uint32_t kOffMisc = kOffWord + 4 * kWStages;
  // + slack to align to 1024 from the 128 that the declaration gives
  static constexpr uint32_t kSmemBytes = kOffMisc + 8 + 896;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};
// Of the launch's 512 x 128 registers (e4m3; bf16 384 x 168) the softmax
// warpgroups take 176 a thread and the other warps keep 80: 256 * 176 + 256 * 80 = 65536.
constexpr int kRegsSoftmax = 176, kRegsOther = 80;
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax) : "memory");
}
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther) : "memory");
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(r));
}
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void named_bar_sync(int id, int nthreads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}
__device__ __forceinline__ void st_shared_zero16(uint32_t a) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0) : "memory");
}

// A K / V tile with an L2 eviction priority.
__device__ __forceinline__ void tma_load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                              int c0, int c1, int c2, int c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
      "l"(policy)
      : "memory");
}

// One look at an mbarrier phase.
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounded wait on an mbarrier phase; false when the CTA aborts or the limit
// passes (then the abort flag and the error bit are set).
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                         int32_t* err, unsigned long long limit_ns,
                                         bool honour_abort = true) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = globaltimer();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (honour_abort && *abort_flag) return false;
      if (globaltimer() - t0 > limit_ns) {
        atomicOr(err, HPC_DEVCHK_TIMEOUT);
        *abort_flag = 1;
        return false;
      }
    }
  }
}

// Several arrivals at once.
__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar),
               "r"(n)
               : "memory");
}
__device__ __forceinline__ void st_release_word(uint32_t addr, uint32_t v) {
  asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// Bounded wait until the producer has issued tile `tile` into its slot. A slot's
// successive rounds go to different warps, so a warp may ask for round r while
// the slot's barrier has completed only round r - 2, which the parity cannot
// tell apart. Once the slot's word equals the tile, rounds < r are complete and
// round r + 1 cannot start before this warp lets go, so the parity wait that
// follows is exact.
__device__ __forceinline__ bool wait_word(uint32_t word, uint32_t tile, volatile int* abort_flag,
                                          int32_t* err, unsigned long long limit_ns) {
  const unsigned long long t0 = globaltimer();
  for (uint32_t it = 1;; ++it) {
    uint32_t v;
    asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(word) : "memory");
    if (v == tile) return true;
    if ((it & 63u) == 0) {
      if (*abort_flag) return false;
      if (globaltimer() - t0 > limit_ns) {
        atomicOr(err, HPC_DEVCHK_TIMEOUT);
        *abort_flag = 1;
        return false;
      }
    }
  }
}

// The maximum that a state leaves with: -inf for a row without a visible key
// (the merge then skips its o), and a finite one where the scores were NaN only,
// which the maximum has passed over, so that the NaN in l and o are not skipped.
__device__ __forceinline__ float state_max(float m, float l) {
  return l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m);
}

// One piece: tiles [tb, te) of (work row v, KV head h).
struct Piece {
  int h, tb, te;
  bool two;  // two row tiles
};

// The pieces of a part, in order; every role walks the same ones. The next
// work row's record is loaded one row ahead.
struct Walk {
  const int4* recs;
  int v, u, h, v1, u1, H;  // h: the KV head of unit u, kept beside it: no division per piece
  int4 ra, rb, na, nb;  // records of rows v and v + 1: {pair0, pairs, table, tile0}, {tiles, own, len, -}
  __device__ __forceinline__ void load(int row, int4& a, int4& b) const {
    a = recs[2 * row];
    b = recs[2 * row + 1];
  }
  __device__ __forceinline__ bool has(int row) const { return row < v1 || (row == v1 && u1 > 0); }
  __device__ void begin(const PrefixParams& p, int part) {
    const int2* bounds = reinterpret_cast<const int2*>(p.words + p.bound_off);
    recs = reinterpret_cast<const int4*>(p.words + p.rec_off);
    H = p.num_kv_heads;
    // the part's boundaries and its first record in one trip (a plan without
    // units has all boundaries behind the last row)
    const int2 b0 = bounds[part], b1 = bounds[part + 1];
    const int4* first = reinterpret_cast<const int4*>(p.words + p.first_off) + 2 * part;
    ra = first[0];
    rb = first[1];
    na = nb = make_int4(0, 0, 0, 0);
    v = b0.x;
    u = b0.y;
    v1 = b1.x;
    u1 = b1.y;
    h = rb.x > 0 ? u / rb.x : 0;
    if (has(v + 1)) load(v + 1, na, nb);
  }
  __device__ __forceinline__ bool next(Piece& s) {
    while (v < v1 || (v == v1 && u < u1)) {
      const int n = rb.x, all = H * n, end = v == v1 ? min(u1, all) : all;
      if (u < end) {
        const int first = h * n;
        s.h = h;
        s.tb = u - first;
        s.te = min(first + n, end) - first;
        s.two = ra.y > kPrefixTilePairs;
        u = first + s.te;
        h += s.te == n;
        return true;
      }
      ++v;
      u = h = 0;
      ra = na;
      rb = nb;
      if (has(v + 1)) load(v + 1, na, nb);
    }
    return false;
  }
};

template <bool FP8>
__global__ void __launch_bounds__(Lay<FP8>::kThreads, 1)
    prefix_decode_kernel(const __grid_constant__ PrefixParams p,
                         const __grid_constant__ CUtensorMap tmq16,
                         const __grid_constant__ CUtensorMap tmqt,
                         const __grid_constant__ CUtensorMap tmk,
                         const __grid_constant__ CUtensorMap tmv) {
  using Lt = Lay<FP8>;
  constexpr int S = Lt::kStages, S8 = Lt::kStages8;
  constexpr int S8n = S8 > 0 ? S8 : 1;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // 128-byte swizzle atoms need 1024-B alignment
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t sQ = base + Lt::kOffQ, sKV = base + Lt::kOffKV, sKV8 = base + Lt::kOffKV8;
  const uint32_t bars = base + Lt::kOffBar;
  auto q_full = [&](int i) { return bars + 8u * i; };
  auto q_empty = [&](int i) { return bars + 8u * (2 + i); };
  auto q_ready = [&](int i) { return bars + 8u * (4 + i); };  // FP8: Q slot i converted
  auto kv_full = [&](int s) { return bars + 8u * (6 + s); };
  auto kv_empty = [&](int s) { return bars + 8u * (6 + S + s); };
  auto kv8_full = [&](int s) { return bars + 8u * (6 + 2 * S + s); };
  auto kv8_empty = [&](int s) { return bars + 8u * (6 + 2 * S + S8 + s); };
  const uint32_t x_full = bars + 8u * (6 + 2 * S + 2 * S8), x_free = x_full + 8u;
  auto dep_full = [&](int i) { return x_full + 16u + 8u * i; };  // warp pieces' states
  auto dep_free = [&](int i) { return x_full + 32u + 8u * i; };
  const uint32_t q_done = x_full + 48u;  // the last MMA on a Q slot is done
  auto gbar = [&](int g, int k) { return x_full + 56u + 8u * (7 * g + k); };
  auto s_full = [&](int g, int i) { return gbar(g, i); };
  auto p_full = [&](int g, int i) { return gbar(g, 2 + i); };
  auto pv_done = [&](int g, int i) { return gbar(g, 4 + i); };
  auto drain = [&](int g) { return gbar(g, 6); };
  auto w_full = [&](int s) { return FP8 ? gbar(2, s) : kv_full(s); };  // warp pieces
  auto w_empty = [&](int s) { return FP8 ? gbar(2, Lt::kWStages + s) : kv_empty(s); };
  volatile int8_t* s_exp = reinterpret_cast<volatile int8_t*>(smem + Lt::kOffScale);  // Q scales
  volatile float* s_x = reinterpret_cast<volatile float*>(smem + Lt::kOffX);  // m, l of pipeline 1
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + Lt::kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + Lt::kOffMisc + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = blockIdx.x;
  const unsigned long long lim_ns = p.timeout_ns;
  int32_t* err = p.err;
  auto wait = [&](uint32_t bar, uint32_t phase) {
    return wait_bar(bar, phase & 1u, s_abort, err, lim_ns);
  };
  auto wait_all = [&](uint32_t bar, uint32_t phase) {
    return __all_sync(0xffffffffu, wait_bar(bar, phase & 1u, s_abort, err, lim_ns)) != 0;
  };

  if (warp == Lt::kProducerWarp) {
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(q_full(i), 1);
        mbar_init(q_empty(i), 2);  // one arrival per MMA warp
        mbar_init(q_ready(i), kRows);
      }
      for (int s = 0; s < S; ++s) {
        mbar_init(kv_full(s), FP8 ? 32 * Lt::kConvWarps : 1);
        mbar_init(kv_empty(s), 2);  // one arrival per MMA warp
      }
      for (int s = 0; s < S8; ++s) {
        mbar_init(kv8_full(s), 1);
        mbar_init(kv8_empty(s), 32 * Lt::kConvWarps);
      }
      mbar_init(x_full, kRows);
      mbar_init(x_free, kRows);
      for (int i = 0; i < 2; ++i) {
        mbar_init(dep_full(i), 8);  // one arrival per softmax warp
        mbar_init(dep_free(i), 1);
      }
      mbar_init(q_done, 2);  // one commit per MMA warp
      for (int s = 0; s < Lt::kWStages; ++s) {
        st_release_word(base + Lt::kOffWord + 4 * s, 0xFFFFFFFFu);
        if (FP8) {
          mbar_init(w_full(s), 1);
          mbar_init(w_empty(s), 1);
        }
      }
      for (int g = 0; g < 2; ++g) {
        for (int i = 0; i < 2; ++i) {
          mbar_init(s_full(g, i), 1);
          mbar_init(p_full(g, i), kRows);
          mbar_init(pv_done(g, i), 1);
        }
        mbar_init(drain(g), 1);
      }
      *s_abort = 0;
      fence_barrier_init();
      prefetch_map(&tmq16);
      prefetch_map(&tmqt);
      prefetch_map(&tmk);
      prefetch_map(&tmv);
    }
  } else if (warp == Lt::kMmaWarp0) {
    tmem_alloc(smem_u32(s_tmem), 2 * kColsPerPipe);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();  // the plan (and inputs) of the preceding kernels are visible
  griddep_launch_dependents();
  const uint32_t tmem = *s_tmem;
  // one new token per sequence: own pieces (they come after all shared ones) are
  // warp pieces
  const bool warp_own = p.q_len == 1;

  // Each role begins its walk behind its register split: one that lives across it
  // was kept in local memory (e4m3: 71.2 -> 65.1 us).
  Walk walk;
  Piece pc;
  int uses[2] = {0, 0};  // fills of each Q slot before this piece
  int ones = 0;          // one-row-tile pieces before this one (their Q slots alternate)
  int kt = 0;            // K / V tiles of the ring before this piece
  int kw = 0;            // FP8: the same, of the warp pieces' ring

  if (warp == Lt::kProducerWarp) {
    // ------------------------------------------------------------ producer
    regs_dec();
    walk.begin(p, part);
    uint64_t read_once, shared_tiles;  // own tiles leave L2 first: row tiles read shared ones again
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(read_once));
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(shared_tiles));
    int issued = 0, issued_w = 0;                 // K / V tiles issued, in order
    int q_issued[2] = {0, 0};                     // fills issued per Q slot
    int stop = p.withhold_copies != 0 ? 1 : 0;    // failure-path test: nothing is issued
    while (!stop && walk.next(pc)) {
      const int n = pc.te - pc.tb, pair0 = walk.ra.x, table = walk.ra.z;
      const int tile0 = walk.ra.w + pc.tb;
      const bool own = walk.rb.y != 0;
      const int c1 = p.kv_swap ? pc.h : 0, c2 = p.kv_swap ? 0 : pc.h;
      const int slot0 = pc.two ? 0 : (ones & 1), slot1 = pc.two ? 1 : slot0;
      for (int sl = slot0; sl <= slot1 && !(own && warp_own); ++sl) {
        if (lane == 0 && !stop) {
          const int fill = uses[sl];
          if (fill == 0 || wait(q_empty(sl), fill - 1)) {
            const uint32_t dq = sQ + (uint32_t)sl * kQSlotBytes;
            const int row = pair0 + (pc.two ? kPrefixTilePairs * sl : 0);
            // own rows: exactly the q_len pairs; rows past them stay as they are
            const CUtensorMap* map = own ? &tmqt : &tmq16;
            const uint32_t bytes =
                own ? kQSlotBytes / kPrefixTilePairs * (uint32_t)p.q_len : kQSlotBytes;
            mbar_expect_tx(q_full(sl), bytes);
            tma_load_3d(dq, map, q_full(sl), 0, kGroupRows * pc.h, row);
            tma_load_3d(dq + kQHalfBytes, map, q_full(sl), 64, kGroupRows * pc.h, row);
            q_issued[sl] = fill + 1;
          } else {
            stop = 1;
          }
        }
        ++uses[sl];
      }
      if (!pc.two) ++ones;
      stop = __shfl_sync(0xffffffffu, stop, 0);
      const bool to_warps = FP8 && own && warp_own;
      const uint64_t policy = own ? read_once : shared_tiles;
      if (to_warps && kw == 0) {
        // the warp pieces' ring lies over the two others: every MMA on them is done
        if (lane == 0 && !wait(q_done, 0)) stop = 1;
        stop = __shfl_sync(0xffffffffu, stop, 0);
      }
      const int32_t* btrow = p.block_table + (int64_t)table * p.bt_sb;
      for (int j0 = 0; j0 < n && !stop; j0 += 32) {
        int blk = -1;  // out of range: TMA fills zeros
        if (j0 + lane < n) {
          const int jj = tile0 + j0 + lane;
          if (jj < p.max_blocks) {
            const int x = __ldg(btrow + jj);
            if (x >= 0 && x < p.num_blocks) blk = x;
            else atomicOr(err, HPC_DEVCHK_BAD_BLOCK);
          } else {
            atomicOr(err, HPC_DEVCHK_TABLE_TOO_SHORT);
          }
        }
        const int cnt = min(n - j0, 32);
        for (int q = 0; q < cnt; ++q) {
          const int bk = __shfl_sync(0xffffffffu, blk, q);
          if (lane == 0) {
            const int j = (to_warps ? kw : kt) + j0 + q;
            if (to_warps) {
              const int slot = j % Lt::kWStages, round = j / Lt::kWStages;
              if (round == 0 || wait(w_empty(slot), round - 1)) {
                st_release_word(base + Lt::kOffWord + 4 * slot, (uint32_t)j);
                const uint32_t dk = sKV + slot * kStageBytes8;
                mbar_expect_tx(w_full(slot), kStageBytes8);
                tma_load_tile(dk, &tmk, w_full(slot), 0, c1, c2, bk, policy);
                tma_load_tile(dk + kKVTileBytes8, &tmv, w_full(slot), 0, c1, c2, bk, policy);
                issued_w = j + 1;
              } else {
                stop = 1;
              }
            } else if (FP8) {
              const int slot = j % S8n, round = j / S8n;
              if (round == 0 || wait(kv8_empty(slot), round - 1)) {
                const uint32_t fb = kv8_full(slot);
                const uint32_t dk = sKV8 + slot * kStageBytes8, dv = dk + kKVTileBytes8;
                mbar_expect_tx(fb, kStageBytes8);
                tma_load_tile(dk, &tmk, fb, 0, c1, c2, bk, policy);
                tma_load_tile(dv, &tmv, fb, 0, c1, c2, bk, policy);
                issued = j + 1;
              } else {
                stop = 1;
              }
            } else {
              const int slot = j % S, round = j / S;
              if (round == 0 || wait(kv_empty(slot), round - 1)) {
                const uint32_t fb = kv_full(slot);
                st_release_word(base + Lt::kOffWord + 4 * slot, (uint32_t)j);
                const uint32_t dk = sKV + slot * kStageBytes, dv = dk + kKVTileBytes;
                mbar_expect_tx(fb, kStageBytes);
                tma_load_tile(dk, &tmk, fb, 0, c1, c2, bk, policy);
                tma_load_tile(dk + kKVTileBytes / 2, &tmk, fb, 64, c1, c2, bk, policy);
                tma_load_tile(dv, &tmv, fb, 0, c1, c2, bk, policy);
                tma_load_tile(dv + kKVTileBytes / 2, &tmv, fb, 64, c1, c2, bk, policy);
                issued = j + 1;
              } else {
                stop = 1;
              }
            }
          }
          stop = __shfl_sync(0xffffffffu, stop, 0);
          if (stop) break;
        }
      }
      if (to_warps) kw += n;
      else kt += n;
    }
    named_bar_sync(1, Lt::kThreads);
    // drain: the last copy issued into each ring slot and each Q slot has landed
    if (lane == 0) {
      constexpr int SR = FP8 ? S8n : S;  // the ring the copies went to
      for (int s = 0; s < SR && s < issued; ++s) {
        const int rounds = (issued - s + SR - 1) / SR;
        wait_bar(FP8 ? kv8_full(s) : kv_full(s), (rounds - 1) & 1, s_abort, err, lim_ns, false);
      }
      for (int s = 0; s < Lt::kWStages && s < issued_w; ++s) {
        const int rounds = (issued_w - s + Lt::kWStages - 1) / Lt::kWStages;
        wait_bar(w_full(s), (rounds - 1) & 1, s_abort, err, lim_ns, false);
      }
      for (int i = 0; i < 2; ++i)
        if (q_issued[i] > 0)
          wait_bar(q_full(i), (q_issued[i] - 1) & 1, s_abort, err, lim_ns, false);
    }
  } else if (FP8 && warp >= Lt::kConvWarp0 && warp < Lt::kProducerWarp) {
    // -------------------------------------------- e4m3 -> f16 converters
    // Each e4m3 tile (64 token rows x 128 bytes, 128-byte swizzle: 16-byte
    // chunk c of row t at c ^ (t % 8)) is widened exactly into the f16 tile the
    // MMAs read (two 64-column halves, 8-element chunk c' of row t at
    // c' ^ (t % 8)). Each group of 8 threads serving one 16-byte access covers
    // all 8 bank groups on the load and both stores. V rows behind the end of
    // the sequence become zeros.
    regs_dec();
    walk.begin(p, part);
    constexpr int kNT = 128;
    const int ct = threadIdx.x - 32 * Lt::kConvWarp0;
    const int cq = ct & 15, c = cq & 7, cr = ((cq >> 2) & 1) ^ (cq >> 3);
    bool ok = true;
    while (ok && walk.next(pc)) {
      if (walk.rb.y && warp_own) break;  // the e4m3 tiles of warp pieces are read as they are
      const int n = pc.te - pc.tb;
      const int len = walk.rb.y ? walk.rb.z : INT32_MAX, tile0 = walk.ra.w + pc.tb;
      for (int j = 0; ok && j < n; ++j) {
        const int k = kt + j, s8 = k % S8n, sb = k % S;
        ok = wait_all(kv8_full(s8), k / S8n);
        if (ok && k >= S) ok = wait_all(kv_empty(sb), k / S - 1);
        if (!ok) break;
        const int valid = len - (tile0 + j) * kBlockTokens;  // rows of this tile that exist
        const uint32_t e8 = sKV8 + s8 * kStageBytes8, kb = sKV + sb * kStageBytes;
#pragma unroll
        for (int it0 = 0; it0 < 1024 / kNT; it0 += 4) {  // four loads in flight per thread
          uint32_t xs[4][4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int t = u * 16 + (ct >> 4) * 2 + cr;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(xs[u][0]), "=r"(xs[u][1]), "=r"(xs[u][2]), "=r"(xs[u][3])
                         : "r"(e8 + (it0 >> 2) * kKVTileBytes8 + t * 128 +
                               ((uint32_t)(c ^ (t & 7)) << 4)));
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int t = u * 16 + (ct >> 4) * 2 + cr;
            uint32_t w[8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              w[2 * q] = e4m3x2_to_f16x2(xs[u][q]);
              w[2 * q + 1] = e4m3x2_to_f16x2(xs[u][q] >> 16);
            }
            const int cc = (c & 3) * 2;
            const uint32_t row =
                kb + (it0 >> 2) * kKVTileBytes + (c >> 2) * (kKVTileBytes / 2) + t * 128;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             row + ((uint32_t)(cc ^ (t & 7)) << 4)),
                         "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                         : "memory");
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             row + ((uint32_t)((cc + 1) ^ (t & 7)) << 4)),
                         "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                         : "memory");
          }
        }
        if (valid < kBlockTokens) {  // V rows behind the sequence's end: this thread's chunks
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int t = u * 16 + (ct >> 4) * 2 + cr, cc = (c & 3) * 2;
            const uint32_t row = kb + kKVTileBytes + (c >> 2) * (kKVTileBytes / 2) + t * 128;
            if (t >= valid) {
              st_shared_zero16(row + ((uint32_t)(cc ^ (t & 7)) << 4));
              st_shared_zero16(row + ((uint32_t)((cc + 1) ^ (t & 7)) << 4));
            }
          }
        }
        fence_async_shared();  // the MMAs read the f16 tile through the async proxy
        mbar_arrive(kv8_empty(s8));
        mbar_arrive(kv_full(sb));
      }
      kt += n;
    }
    named_bar_sync(1, Lt::kThreads);
  } else if (warp >= Lt::kMmaWarp0 + 2) {
    regs_dec();  // the idle warp of the last warpgroup
    named_bar_sync(1, Lt::kThreads);
  } else if (warp >= Lt::kMmaWarp0) {
    // ------------------------------------------- MMA issue for pipeline g
    // The whole warp runs the schedule so its values stay warp-uniform; one
    // elected lane issues the MMAs and commits.
    regs_dec();
    walk.begin(p, part);
    const int g = warp - Lt::kMmaWarp0;
    const bool leader = elect_one() != 0;
    bool issued_any = false;
    constexpr uint32_t kIdS =
        FP8 ? idesc_f16_f32(kRows, 64, false, false) : idesc_bf16_f32(kRows, 64, false, false);
    constexpr uint32_t kIdPV =
        FP8 ? idesc_f16_f32(kRows, 128, false, true) : idesc_bf16_f32(kRows, 128, false, true);
    const uint64_t kd0 = smem_desc_sw128(sKV, 16, 1024);
    // V: MN-major; 64-column halves 8 KB apart, 8-token row groups 1 KB apart
    const uint64_t vd0 = smem_desc_sw128(sKV + kKVTileBytes, kKVTileBytes / 2, 1024);
    const uint32_t dS = tmem + kColsPerPipe * g + kColS, od = tmem + kColsPerPipe * g + kColO;
    // The end of a warp piece (warp pieces of parity g are this warp's): the
    // states of the 8 softmax warps joined, in warp order, and written out.
    auto finish_warp_piece = [&](int use) -> bool {
      if (!wait_all(dep_full(g), use)) return false;
      const int d8 = lane >> 2, h2 = 2 * (lane & 3);  // accumulator lane: rows d8, heads h2, h2 + 1
      const volatile float* ml = s_x + g * kRows;     // [8 warps][m of 8 heads, l of 8 heads]
      float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        M0 = fmaxf(M0, ml[16 * w + h2]);
        M1 = fmaxf(M1, ml[16 * w + h2 + 1]);
      }
      float l0 = 0.f, l1 = 0.f, acc[8][4];
#pragma unroll
      for (int dm = 0; dm < 8; ++dm) acc[dm][0] = acc[dm][1] = acc[dm][2] = acc[dm][3] = 0.f;
#pragma unroll 2
      for (int w = 0; w < 8; ++w) {
        const float m0 = ml[16 * w + h2], m1 = ml[16 * w + h2 + 1];
        if (m0 == -INFINITY && ml[16 * w + 8 + h2] == 0.f) continue;  // no tile in this piece
        const float f0 = ex2(m0 - M0), f1 = ex2(m1 - M1);
        l0 += ml[16 * w + 8 + h2] * f0;
        l1 += ml[16 * w + 9 + h2] * f1;
        const uint32_t src = sQ + (uint32_t)g * kQSlotBytes + (uint32_t)w * 4096u + 16u * lane;
#pragma unroll
        for (int dm = 0; dm < 8; ++dm) {
          float a, b, c2, d2;
          asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(a), "=f"(b), "=f"(c2), "=f"(d2)
                       : "r"(src + 512u * dm));
          acc[dm][0] += a * f0;
          acc[dm][1] += b * f1;
          acc[dm][2] += c2 * f0;
          acc[dm][3] += d2 * f1;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(dep_free(g));
      const int64_t blk = pc.tb == 0
                              ? p.ws.own0 + (int64_t)walk.ra.x * p.num_kv_heads + pc.h
                              : p.ws.cont0 + (int64_t)part * kPrefixRowPairs;
      float* dst = reinterpret_cast<float*>(p.ws.o + blk * 256);  // [d / 4][head][d % 4]
#pragma unroll
      for (int dm = 0; dm < 8; ++dm)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int d = acc_d<FP8>(dm, r, d8);
          dst[(d >> 2) * 32 + 4 * h2 + (d & 3)] = acc[dm][2 * r];
          dst[(d >> 2) * 32 + 4 * h2 + 4 + (d & 3)] = acc[dm][2 * r + 1];
        }
      if (lane < 4) {
        p.ws.m[blk * 8 + h2] = state_max(M0, l0);
        p.ws.m[blk * 8 + h2 + 1] = state_max(M1, l1);
        p.ws.l[blk * 8 + h2] = l0;
        p.ws.l[blk * 8 + h2 + 1] = l1;
      }
      return true;
    };
    int c = 0;  // tiles of this pipeline before this piece
    int warp_pieces = 0;
    bool ok = true;
    while (ok && walk.next(pc)) {
      const int n = pc.te - pc.tb;
      if (walk.rb.y && warp_own) {
        if (warp_pieces == 0 && leader) mma_commit(q_done);
        __syncwarp();
        if ((warp_pieces & 1) == g) ok = finish_warp_piece(warp_pieces >> 1);
        ++warp_pieces;
        continue;
      }
      const int slot0 = pc.two ? 0 : (ones & 1), slot1 = pc.two ? 1 : slot0;
      const int my_slot = pc.two ? g : slot0;
      const int stride = pc.two ? 1 : 2, first = pc.two ? 0 : g;
      const int mine = first < n ? (n - first + stride - 1) / stride : 0;  // tiles of this pipeline
      // S(i) = Q K^T for the pipeline's i-th tile of the piece, into the S buffer
      // of its parity. That held P of the tile two before, whose P V this thread
      // has issued earlier: the tensor pipe runs them in order.
      const uint64_t qd = smem_desc_sw128(sQ + (uint32_t)my_slot * kQSlotBytes, 16, 1024);
      auto issue_s = [&](int i) {
        const int slot = (kt + first + i * stride) % S;
        tc_fence_after();
        const uint64_t kd = kd0 + (uint64_t)(slot * (kStageBytes >> 4));
        const uint32_t d = dS + 64u * (uint32_t)((c + i) & 1);
        if (leader) {
          // Q and K: K-major; 64-column halves 16 KB / 8 KB apart, 16 columns = 32 bytes
          mma_f16_ss(d, qd, kd, kIdS, 0u);
#pragma unroll
          for (int kk = 1; kk < 8; ++kk)
            mma_f16_ss(d, qd + (kk >> 2) * (kQHalfBytes >> 4) + (kk & 3) * 2,
                       kd + (kk >> 2) * ((kKVTileBytes / 2) >> 4) + (kk & 3) * 2, kIdS, 1u);
          mma_commit(s_full(g, (c + i) & 1));
          if (i + 1 == mine) mma_commit(q_empty(my_slot));
        }
        __syncwarp();
      };
      // O += P V for the i-th tile, P from tensor memory (16 keys = 8 columns
      // per step); the ring slot is released once the MMAs on it are done
      auto issue_pv = [&](int i) {
        const int k = kt + first + i * stride, x = c + i;
        tc_fence_after();
        const uint64_t vd = vd0 + (uint64_t)((k % S) * (kStageBytes >> 4));
        const uint32_t pa = tmem + kColsPerPipe * g + kColS + 64u * (uint32_t)(x & 1);
        if (leader) {
          mma_f16_ts(od, pa, vd, kIdPV, i > 0 ? 1u : 0u);
#pragma unroll
          for (int kk = 1; kk < 4; ++kk) mma_f16_ts(od, pa + 8 * kk, vd + kk * (2048 >> 4), kIdPV, 1u);
          mma_commit(pv_done(g, x & 1));
          mma_commit(kv_empty(k % S));
        }
        __syncwarp();
      };
      // Q as landed (BF16) or converted (FP8); a slot that this pipeline does
      // not use gets its arrival once it is filled
      for (int sl = slot0; ok && sl <= slot1; ++sl) {
        ok = wait_all(FP8 ? q_ready(sl) : q_full(sl), uses[sl]);
        if (ok && (sl != my_slot || mine == 0)) {
          if (leader) mbar_arrive(q_empty(sl));
          __syncwarp();
        }
        ++uses[sl];
      }
      if (!pc.two) ++ones;
      // Whatever is ready next. The ring's tiles in their order (a look at a later
      // slot's barrier could see a stale phase): S(s) for this pipeline's, whose
      // buffer is free once P V(s - 2) is issued; for the other pipeline's, with
      // one row tile, this warp's arrival once the tile has landed. And P V(v).
      int s = 0, v = 0, j = 0;  // S and P V issued, tiles of the ring passed
      unsigned long long idle_since = 0;
      for (uint32_t it = 1; ok && (v < mine || j < n);) {
        bool did = false;
        const bool own_tile = stride == 1 || (j & 1) == g;
        if (j < n && (!own_tile || s < v + 2)) {
          const int k = kt + j;
          if (__all_sync(0xffffffffu, mbar_test_wait(kv_full(k % S), (k / S) & 1))) {
            if (own_tile) {
              issue_s(s++);
              issued_any = true;
            } else {
              if (leader) mbar_arrive(kv_empty(k % S));
              __syncwarp();
            }
            ++j;
            did = true;
          }
        }
        if (v < s && __all_sync(0xffffffffu,
                                mbar_test_wait(p_full(g, (c + v) & 1), ((c + v) >> 1) & 1))) {
          issue_pv(v++);
          did = true;
        }
        if (did) {
          idle_since = 0;
        } else if ((++it & 63u) == 0) {  // bounded: nothing ready for the limit
          const unsigned long long now = globaltimer();
          if (idle_since == 0) idle_since = now;
          const bool late = now - idle_since > lim_ns;
          if (__any_sync(0xffffffffu, late || *s_abort)) {
            if (late && lane == 0) {
              atomicOr(err, HPC_DEVCHK_TIMEOUT);
              *s_abort = 1;
            }
            ok = false;
          }
        }
      }
      c += mine;
      kt += n;
    }
    if (leader && issued_any) {
      mma_commit(drain(g));  // every MMA this lane issued has completed
      wait_bar(drain(g), 0, s_abort, err, lim_ns, false);
    }
    __syncwarp();
    tc_fence_before();
    named_bar_sync(1, Lt::kThreads);
    tc_fence_after();
    if (warp == Lt::kMmaWarp0) tmem_dealloc(tmem, 2 * kColsPerPipe);
  } else {
    // ------------------------------------------- softmax warpgroup of pipeline g
    regs_inc();
    walk.begin(p, part);
    const int g = warp >> 2;
    const int r = threadIdx.x - kRows * g;  // query row = TMEM lane
    const int wg_warp = warp & 3;
    const uint32_t lanes = (uint32_t)(wg_warp * 32) << 16;
    const uint32_t trow = tmem + kColsPerPipe * g + lanes;
    const int T = p.q_len;
    int cnt_of[2] = {0, 0};  // tiles of each pipeline before this piece
    int joins = 0;           // pieces whose two states were joined, before this one
    int warp_pieces = 0;
    bool ok = true;
    while (ok && walk.next(pc)) {
      const int n = pc.te - pc.tb;
      if (walk.rb.y && warp_own) {
        // ---- warp piece: this warp takes every 8th tile of the ring
        float acc[8][4];
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int dm = 0; dm < 8; ++dm) acc[dm][0] = acc[dm][1] = acc[dm][2] = acc[dm][3] = 0.f;
        const int k0 = FP8 ? kw : kt;  // the piece's first tile in its ring
        const int j0 = (warp - k0) & 7;
        if (j0 < n) {
          uint32_t qf[8][2];
          const float sl2 =
              p.score_scale_log2 * load_q<FP8>(p.q + (int64_t)walk.ra.x * p.q_sp +
                                                   (int64_t)(kGroupRows * pc.h) * p.q_sh,
                                               p.q_sh, lane, qf);
          for (int j = j0; j < n; j += 8) {
            const int k = k0 + j, slot = k % Lt::kWStages;
            ok = __all_sync(0xffffffffu, wait_word(base + Lt::kOffWord + 4 * slot, (uint32_t)k,
                                                   s_abort, err, lim_ns));
            if (ok) ok = wait_all(w_full(slot), k / Lt::kWStages);
            if (!ok) break;
            const uint32_t kb = sKV + slot * Lt::kWStageBytes;
            const uint32_t vb = kb + Lt::kWStageBytes / 2;
            const int valid = walk.rb.z - (walk.ra.w + pc.tb + j) * kBlockTokens;
            if (valid < kBlockTokens) {
              // V rows behind the sequence's end (both column halves of a 16-bit tile)
              constexpr int kHalves = FP8 ? 1 : 2;
              for (int q = lane; q < (kBlockTokens - valid) * 8 * kHalves; q += 32)
                st_shared_zero16(vb + (q & 8) / 8 * (kHalves - 1) * (kKVTileBytes / 2) +
                                 (uint32_t)(valid + q / (8 * kHalves)) * 128 +
                                 (uint32_t)(q & 7) * 16);
              __syncwarp();
            }
            compute_unit<FP8>(kb, vb, qf, valid, sl2, m, l, acc, lane);
            if (valid < kBlockTokens) fence_async_shared();  // before TMA writes there again
            __syncwarp();
            if (lane == 0) mbar_arrive_n(w_empty(slot), FP8 ? 1 : 2);  // (both MMA warps' arrivals)
          }
          if (!ok) break;
        }
        // the state of this warp to the piece's buffer; the warp that joins them
        // is the MMA warp of the buffer's number
        const int buf = warp_pieces & 1, use = warp_pieces >> 1;
        if (use > 0) {
          ok = wait_all(dep_free(buf), use - 1);
        } else {
          // first use: the buffers lie in the Q slots and the join cells
          ok = wait_all(q_done, 0);
          if (ok && joins > 0) ok = wait_all(x_free, joins - 1);
        }
        if (!ok) break;
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
          l[1] += __shfl_xor_sync(0xffffffffu, l[1], o);
        }
        volatile float* ml = s_x + buf * kRows + 16 * warp;
        if (lane < 4) {
          ml[2 * lane] = m[0];
          ml[2 * lane + 1] = m[1];
          ml[8 + 2 * lane] = l[0];
          ml[9 + 2 * lane] = l[1];
        }
        if (j0 < n) {
          const uint32_t dst = sQ + (uint32_t)buf * kQSlotBytes + (uint32_t)warp * 4096u + 16u * lane;
#pragma unroll
          for (int dm = 0; dm < 8; ++dm)
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dst + 512u * dm),
                         "f"(acc[dm][0]), "f"(acc[dm][1]), "f"(acc[dm][2]), "f"(acc[dm][3])
                         : "memory");
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(dep_full(buf));
        ++warp_pieces;
        if (FP8) kw += n;
        else kt += n;
        continue;
      }
      const int slot0 = pc.two ? 0 : (ones & 1);
      const int my_slot = pc.two ? g : slot0;
      const int stride = pc.two ? 1 : 2, first = pc.two ? 0 : g;
      int mine_of[2];
      mine_of[0] = pc.two ? n : (n + 1) / 2;
      mine_of[1] = pc.two ? n : n / 2;
      const int mine = g == 0 ? mine_of[0] : mine_of[1];
      const int c = g == 0 ? cnt_of[0] : cnt_of[1];
      const int pairs = pc.two && g == 1 ? walk.ra.y - kPrefixTilePairs
                                         : min(walk.ra.y, kPrefixTilePairs);
      const bool row_ok = (r >> 3) < pairs;
      // warps without a row keep the barrier counts only (their S, P and O rows
      // are never read)
      const bool live = 32 * wg_warp < kGroupRows * pairs;
      const int tile0 = walk.ra.w + pc.tb;
      // own tiles: the sequence's last q_len positions are the new tokens, and
      // token t of them sees positions < len - (T - 1 - t)
      const int len = walk.rb.y ? walk.rb.z : INT32_MAX;
      const int lim = walk.rb.y && row_ok ? len - (T - 1 - (r >> 3)) : INT32_MAX;
      float sc = p.score_scale_log2;
      int fill = 0;  // FP8: fills of this piece's Q slot before it
      if constexpr (FP8) {
        // The Q rows of a slot are converted in place by the warpgroup of the
        // slot's number: f16 with 2^e putting the row's largest |q| in
        // [2^14, 2^15) (exact for every bf16 value that stays normal); 2^-e goes
        // into the row's logit scale. Chunk i of row r in the order i ^ (r % 8),
        // so the 8 rows of one shared-memory wavefront hit 8 bank groups.
        if (my_slot == g) {
          ok = wait_all(q_full(g), g == 0 ? uses[0] : uses[1]);
          if (ok && row_ok) {
            const uint32_t qrow = sQ + (uint32_t)g * kQSlotBytes + (uint32_t)r * 128;
            auto chunk = [&](int i) {
              return qrow + (i >> 3) * kQHalfBytes + ((uint32_t)((i & 7) ^ (r & 7)) << 4);
            };
            uint32_t m2[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              uint32_t x[4];
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                           : "r"(chunk(i)));
#pragma unroll
              for (int e = 0; e < 4; ++e)
                asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m2[e]) : "r"(m2[e]), "r"(x[e]));
            }
            float mq = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mq = fmax3(mq, fabsf(__uint_as_float(m2[e] << 16)),
                         fabsf(__uint_as_float(m2[e] & 0xFFFF0000u)));
            int e2 = 0;
            if (mq > 0.f) {
              e2 = 14 - ((int)((__float_as_uint(mq) >> 23) & 0xFF) - 127);
              e2 = e2 < -100 ? -100 : (e2 > 100 ? 100 : e2);
            }
            // a negative scale turns Q around, so that the scores' factor is positive
            const float qs = __uint_as_float(((uint32_t)(127 + e2) << 23) |
                                             (__float_as_uint(p.score_scale_log2) & 0x80000000u));
            s_exp[(2 * g + ((g == 0 ? uses[0] : uses[1]) & 1)) * kRows + r] = (int8_t)e2;
#pragma unroll 4
            for (int i = 0; i < 16; ++i) {
              uint32_t x[4], y[4];
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                           : "r"(chunk(i)));
#pragma unroll
              for (int e = 0; e < 4; ++e)
                y[e] = pack_f16(__uint_as_float(x[e] << 16) * qs,
                                __uint_as_float(x[e] & 0xFFFF0000u) * qs);
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(chunk(i)), "r"(y[0]),
                           "r"(y[1]), "r"(y[2]), "r"(y[3])
                           : "memory");
            }
            fence_async_shared();  // the S MMAs read Q through the async proxy
          }
          mbar_arrive(q_ready(g));
          if (!ok) break;
        }
        fill = my_slot == 0 ? uses[0] : uses[1];
        if (pc.two || slot0 == 0) ++uses[0];
        if (pc.two || slot0 == 1) ++uses[1];
      }
      if (!pc.two) ++ones;
      float m = -INFINITY, l = 0.f;
      for (int i = 0; ok && i < mine; ++i) {
        const int x = c + i;            // tile of this pipeline
        const int j = first + i * stride;  // tile of the piece
        const int kv0 = (tile0 + j) * kBlockTokens;
        ok = wait_all(s_full(g, x & 1), x >> 1);
        if (!ok) break;
        tc_fence_after();
        // S is there, so the Q rows were converted: their scale comes back out
        // (a factor of 0 would make NaN of masked scores: the least normal number
        // times any score, below 2^31, is 0 to every exponential)
        if (FP8 && i == 0 && row_ok)
          sc = fmaxf(fabsf(sc) * __uint_as_float(
                                     (uint32_t)(127 - s_exp[(2 * my_slot + (fill & 1)) * kRows + r]) << 23),
                     FLT_MIN);
        // the state that this pipeline's first P V of the piece overwrites has
        // been joined into warpgroup 0's
        if (g == 1 && i == 0 && joins > 0) {
          ok = wait_all(x_free, joins - 1);
          if (!ok) break;
        }
        if (!FP8 && len - kv0 < kBlockTokens) {
          // V rows behind the sequence's end
          const int k = kt + j, slot = k % S, valid = len - kv0;
          ok = wait_all(kv_full(slot), k / S);
          if (!ok) break;
          const uint32_t v = sKV + slot * kStageBytes + kKVTileBytes;
          for (int q = r; q < (kBlockTokens - valid) * 16; q += kRows)
            st_shared_zero16(v + (q & 8) / 8 * (kKVTileBytes / 2) +
                             (uint32_t)(valid + (q >> 4)) * 128 + (uint32_t)(q & 7) * 16);
          fence_async_shared();  // the P V MMA reads V through the async proxy
        }
        if (live) {
          const uint32_t ts = trow + kColS + 64u * (uint32_t)(x & 1);
          float s[64];
          tmem_ld32(ts, *reinterpret_cast<float(*)[32]>(&s[0]));
          tmem_ld32(ts + 32, *reinterpret_cast<float(*)[32]>(&s[32]));
          tmem_wait_ld();
          if (kv0 > lim - 64) {  // (kv0 + 64 may pass int32)
#pragma unroll
            for (int q = 0; q < 64; ++q)
              if (kv0 + q >= lim) s[q] = -INFINITY;
          }
          float mx8[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) mx8[q] = s[q];
#pragma unroll
          for (int q = 8; q + 16 <= 64; q += 16)
#pragma unroll
            for (int e = 0; e < 8; ++e) mx8[e] = fmax3(mx8[e], s[q + e], s[q + 8 + e]);
#pragma unroll
          for (int q = 0; q < 8; ++q) mx8[q] = fmaxf(mx8[q], s[56 + q]);
          const float mx = fmaxf(fmax3(mx8[0], mx8[1], mx8[2]),
                                 fmax3(fmax3(mx8[3], mx8[4], mx8[5]), mx8[6], mx8[7]));
          const float m_new = fmaxf(m, mx * sc);
          // move the row maximum only when it grew by more than the threshold
          const bool need = row_ok && i > 0 && m_new > m + kRescaleThreshold;
          const float m_use = (i == 0 || need) ? m_new : m;
          const float alpha = need ? ptx_ex2(m - m_new) : 1.f;
          // a row with no visible key so far keeps m = -inf and P = 0
          const float m_ref = m_use == -INFINITY ? 0.f : m_use;
          uint32_t pk[32];
          const uint64_t sc2 = pack2(sc, sc), nm2 = pack2(-m_ref, -m_ref);
          uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
          for (int q = 0; q < 32; ++q) {
            float x0, x1;
            unpack2(ffma2(pack2(s[2 * q], s[2 * q + 1]), sc2, nm2), x0, x1);
            const float p0 = ptx_ex2(x0), p1 = ptx_ex2(x1);
            acc2[q & 3] = fadd2(acc2[q & 3], pack2(p0, p1));
            pk[q] = FP8 ? pack_f16(p0, p1) : pack_bf16(p0, p1);  // keys 2q (low) and 2q + 1
          }
          float r0, r1;
          unpack2(fadd2(fadd2(acc2[0], acc2[1]), fadd2(acc2[2], acc2[3])), r0, r1);
          l = l * alpha + (r0 + r1);
          m = m_use;
          if (i > 0 && __any_sync(0xffffffffu, need)) {
            // O is stable once the P V of tile x - 1 is done
            ok = wait_all(pv_done(g, (x - 1) & 1), (x - 1) >> 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float o[32];
              tmem_ld32(trow + kColO + q * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= alpha;
              tmem_st32(trow + kColO + q * 32, o);
            }
          }
          tmem_st32(ts, pk);  // over S of this tile, which is in registers
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(p_full(g, x & 1));
      }
      if (!ok) break;
      // ---- epilogue of the piece
      const bool join = !pc.two && n > 1;  // two states of the same rows
      if (!(g == 1 && !pc.two)) {
        // O of the tiles of this piece: this pipeline's, and the other's to join
        const int last = c + mine - 1;
        ok = wait_all(pv_done(g, last & 1), last >> 1);
        float m1 = -INFINITY, l1 = 0.f;
        if (ok && join) {
          const int last1 = cnt_of[1] + mine_of[1] - 1;
          ok = wait_all(x_full, joins) && wait_all(pv_done(1, last1 & 1), last1 >> 1);
          if (ok) {
            m1 = s_x[r];
            l1 = s_x[kRows + r];
          }
        }
        if (!ok) break;
        tc_fence_after();
        const float M = fmaxf(m, m1);
        const float a0 = m == -INFINITY ? 0.f : ptx_ex2(m - M);
        const float a1 = m1 == -INFINITY ? 0.f : ptx_ex2(m1 - M);
        if (live) {
          const int pair = r >> 3;  // of this row tile
          int64_t blk;
          if (pc.tb == 0)
            blk = (walk.rb.y ? p.ws.own0 : 0) +
                  (int64_t)(walk.ra.x + kPrefixTilePairs * (pc.two ? g : 0) + pair) * p.num_kv_heads +
                  pc.h;
          else
            blk = p.ws.cont0 + (int64_t)part * kPrefixRowPairs + kPrefixTilePairs * (pc.two ? g : 0) +
                  pair;
          float4* dst = p.ws.o + blk * 256 + (r & 7);  // [32 column groups][8 heads]
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float o[32];
            tmem_ld32(trow + kColO + q * 32, o);
            if (join) {
              float o1[32];
              tmem_ld32(trow + kColsPerPipe + kColO + q * 32, o1);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = o[e] * a0 + o1[e] * a1;
            } else {
              tmem_wait_ld();
            }
            if (row_ok) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                dst[(q * 8 + e) * 8] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
          }
          if (row_ok) {
            const float lt = join ? l * a0 + l1 * a1 : l;
            p.ws.m[blk * 8 + (r & 7)] = state_max(M, lt);
            p.ws.l[blk * 8 + (r & 7)] = lt;
          }
        }
        if (join) {
          tc_fence_before();
          mbar_arrive(x_free);
        }
      } else if (join) {
        // pipeline 1 of a one-row-tile piece: its state goes to warpgroup 0. The
        // cells were last read before the x_free that this warpgroup has waited
        // for in this piece's first tile.
        s_x[r] = m;
        s_x[kRows + r] = l;
        mbar_arrive(x_full);
      }
      if (join) ++joins;
      cnt_of[0] += mine_of[0];
      cnt_of[1] += mine_of[1];
      kt += n;
    }
    tc_fence_before();
    named_bar_sync(1, Lt::kThreads);
  }
}

template <bool FP8>
cudaError_t launch_tc(const PrefixParams& p, const CUtensorMap& tq16, const CUtensorMap& tqt,
                      const CUtensorMap& tk, const CUtensorMap& tv, int num_parts,
                      cudaStream_t stream) {
  using Lt = Lay<FP8>;
  static std::atomic<uint64_t> configured{0};  // devices whose copy is configured
  const cudaError_t e = once_per_device(configured, [] {
    return cudaFuncSetAttribute(prefix_decode_kernel<FP8>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lt::kSmemBytes);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)num_parts);
  cfg.blockDim = dim3(Lt::kThreads);
  cfg.dynamicSmemBytes = Lt::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix_decode_kernel<FP8>, p, tq16, tqt, tk, tv);
}

}  // namespace

cudaError_t launch_prefix_decode(const PrefixParams& p, const CUtensorMap& tq16,
                                 const CUtensorMap& tqt, const CUtensorMap& tk,
                                 const CUtensorMap& tv, bool fp8, int num_parts,
                                 cudaStream_t stream) {
  return fp8 ? launch_tc<true>(p, tq16, tqt, tk, tv, num_parts, stream)
             : launch_tc<false>(p, tq16, tqt, tk, tv, num_parts, stream);
}

}  // namespace hpc
