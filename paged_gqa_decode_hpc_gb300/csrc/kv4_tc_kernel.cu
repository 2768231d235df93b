// Decode attention of 2 to 8 new tokens per sequence over a 4-bit paged cache on the
// 5th-generation tensor cores (tcgen05).
//
// The 8 q_len query rows of a KV head share every tile. With mma.sync the products alone
// take 64 q_len MMAs of 8 issue cycles a unit, and every two tokens their own conversion of the
// codes; here the codes of a unit are converted once and the products cost no issue slots.
//
// Both products run with the wide side in M, so that few query rows cost little:
//  * S^T[token, row] = K Q^T: M = 128 tokens (two tiles, a step), N = the query rows, K =
//    128. A = K in tensor memory: a converter thread is a token; it reads its 72-byte row,
//    multiplies codes by scales (exact in f16) and stores 64 columns of pairs. 72 bytes are 18
//    words, so the 8-byte reads of 16 rows cover all banks once.
//  * The softmax threads are tokens too: a row's maximum is over threads. They keep a
//    reference per query row in shared memory, which moves only when some score passes it by
//    8 (log2 units; a vote of the group's four warps), so that as a rule a thread subtracts,
//    takes exponentials, adds its own sums and writes its row of P^T (f16) to shared memory.
//  * O^T[d, row] += V^T P^T: M = 128 elements, K = tokens. A = V as the MN-major operand of
//    its converted tile, B = P^T, MN-major as written. O^T stays in tensor memory for a
//    piece (a thread is an element d then) and is rescaled there when references move.
// A piece's states go to memory as a whole (out, lse) or as partial states, which a second
// kernel joins.
//
// Warps: two groups of 4 for the softmax (half of the rows each, and their ends of a piece), 4
// that convert q and K, 8 for V (4 to a tile), and one each for the copies of K and V, the
// issue of either product and the copies of q. Plan, ring and copies are kv4_plan.cuh's. Every
// wait is bounded; after one has run out every role leaves, the MMAs are waited for and tensor
// memory is freed.
//
// What bounds it (31 sequences of 4096 and one of 131072 positions, 8 KV heads; HBM's share is
// 44 us, 780 clk a step): the chain from a step's scores to its P^T, about 1000 clk of waits,
// vote and fences that no row count changes and 15 to 25 a row of the group, on warps that share
// the SM's issue (0.5 to 0.6 a cycle) and its shared memory (2 tokens: 710 wavefronts a step
// for threads, 315 for the MMAs, 144 for the copies; V passes twice) with the conversions.
// 2 tokens take 84 us, 4 take 99, 6 112, 8 128. What it took, 4 and 8 tokens: one softmax
// group and one warp for both products 151 and 203 us; two waits a step in that warp and 8
// warps for V 121 and 182; two groups, a warp for each product 102 and 162; a factor for each
// row (see below) 107 and 153; references and factors in registers 102 and 131; a pair counted
// with 7 units 101 and 128; K's two halves in a loop 99 and 126; the
// warp barrier behind a wait on two barriers 99 and 128. Groups that take alternate steps
// instead of rows were slower (118 and 214: their states need more registers). A wait on two
// barriers takes half of the lanes each, one latency instead of two: with every lane at one and
// then at the other 2 tokens take 103 us, 4 129, 8 165.
#include <cfloat>

#include "kv4_plan.cuh"
#include "tc05.cuh"

namespace hpc {
namespace {

// Units that a pair counts for beside its own, and that a CTA is worth starting for (13 short
// sequences with 8 drafts 26.1 us with 4, 23.5 with 6 to 8; 8 short ones of 2 tokens 12.2 us with
// parts of at least 8 units, 10.7 with 4).
constexpr int kPairCost = 7, kMinPart = 4;
constexpr int kThreads = 768;
constexpr int kKWarp0 = 8, kVWarp0 = 12, kProducerWarp = 20, kScoreWarp = 21, kValueWarp = 22;
// (and the last warp: q)
constexpr int kPieceQ = 4;                  // piece descriptors in flight
constexpr int kPieceReaders = 8 + 4 + 8 + 1 + 1 + 1;
constexpr int kVBufs = 4;                   // converted V tiles: two steps
constexpr uint32_t kVTile = 64 * 128 * 2;   // two 64-element halves of 64 x 128 bytes
constexpr uint32_t kPBuf = 128 * 128;       // P^T of a step: 128 rows (tokens) of 128 bytes
// tensor memory: K (2 x 64 columns), S^T (4 x 64), O^T (64)
constexpr uint32_t kColK = 0, kColS = 128, kColO = 384, kTmemCols = 512;
constexpr float kPassed = 8.f;              // log2 units by which a score may pass its reference

// COLS: query rows that are computed (16, 32, 48 or 64), the MMAs' N.
template <int COLS>
struct Cfg {
  static constexpr uint32_t kQHalf = COLS * 128, kQBuf = 2 * kQHalf;  // rows of 64 elements each
  static constexpr uint32_t kOffV = 0;
  static constexpr uint32_t kOffP = kOffV + kVBufs * kVTile;
  static constexpr uint32_t kOffQ = kOffP + 2 * kPBuf;
  static constexpr uint32_t kOffRing = kOffQ + 2 * kQBuf;
  static constexpr int kFixed = kOffRing + 5120 /* barriers, descriptors, references */ + 1024 + 4 * (kKv4MaxSeqs + 1);
  static constexpr int kStages = (227 * 1024 - kFixed) / (2 * kKv4Tile) < 16 ? (227 * 1024 - kFixed) / (2 * kKv4Tile) : 16;
  static constexpr int kBatch = 4;
  static constexpr uint32_t kOffBar = kOffRing + kStages * 2 * kKv4Tile;
  // full, empty [stages]; piece full, free [4]; K full [2], S full, free [4 each], P full, V
  // full, PV done [2 each]; q landed, free [2 each], full [4]; drains [2]
  static constexpr int kNumBars = 2 * kStages + 2 * kPieceQ + 16 + 8 + 2;
  static constexpr uint32_t kOffDesc = kOffBar + (8 * kNumBars + 15) / 16 * 16;
  static constexpr uint32_t kOffFloat = kOffDesc + kPieceQ * 32;
  // references (true, used), factors, 1 / sums, row maxima or sums of four warps; q's factors of
  // four pieces
  static constexpr uint32_t kFloats = 64 * (4 + 4 + 4);
  static constexpr uint32_t kOffMisc = kOffFloat + 4 * kFloats;
  static constexpr uint32_t kOffPlan = kOffMisc + 256;
  static constexpr uint32_t kSmemBytes = 1024 /* alignment slack */ + kOffPlan;
  static constexpr uint32_t kSmemBytesMax = kSmemBytes + 4 * (kKv4MaxSeqs + 1);
  static_assert(kSmemBytesMax <= 227 * 1024, "shared memory");
  static_assert(kOffFloat + 4 * kFloats + 256 - kOffBar <= 5120, "small arrays");
  static_assert(kStages >= 8, "units ahead");
  static constexpr int kHalf = COLS / 2;  // the rows of a softmax group
  // Registers a thread by warpgroup, of the 80 that the launch gives each: softmax (two; four
  // for each of its rows and what they are made from), K, V (two), others. With 64 rows the
  // others are short of some (spills of a dozen words), and wait most of the time.
  static constexpr int kRegsSoftmax = COLS > 48 ? 152 : 128, kRegsK = COLS > 48 ? 48 : 56,
                       kRegsV = COLS > 48 ? 40 : 56, kRegsOther = COLS > 48 ? 48 : 56;
  static_assert(2 * kRegsSoftmax + kRegsK + 2 * kRegsV + kRegsOther == 6 * 80, "registers");
};
// 8 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_ld8(uint32_t a, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t a, const float* v) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(a),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
               "r"(r[7])
               : "memory");
}
// Sums (or maxima) of l[0 .. N) over the warp's lanes, for rows `at` on, to out[]: each exchange
// halves the rows that a lane goes on with, while they are even.
template <bool MAX, int W, int N, int COLS>
__device__ __forceinline__ void reduce_rows(float (&l)[COLS], int at, float* out, int lane) {
  auto join = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
  if constexpr (W == 0) {
#pragma unroll
    for (int c = 0; c < N; ++c) out[at + c] = l[c];
  } else if constexpr (N % 2 == 0) {
    const bool up = (lane & W) != 0;
#pragma unroll
    for (int c = 0; c < N / 2; ++c) {
      const float give = up ? l[c] : l[c + N / 2];
      l[c] = join(up ? l[c + N / 2] : l[c], __shfl_xor_sync(0xffffffffu, give, W));
    }
    reduce_rows<MAX, W / 2, N / 2>(l, up ? at + N / 2 : at, out, lane);
  } else {
#pragma unroll
    for (int c = 0; c < N; ++c) l[c] = join(l[c], __shfl_xor_sync(0xffffffffu, l[c], W));
    reduce_rows<MAX, W / 2, N>(l, at, out, lane);
  }
}

template <int COLS>
__global__ void __launch_bounds__(kThreads, 1)
    kv4_tc_kernel(const __grid_constant__ Kv4DecodeParams p, const __grid_constant__ CUtensorMap tmq) {
  using C = Cfg<COLS>;
  constexpr int R = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t base = smem_u32(smem);
  const uint32_t bars = base + C::kOffBar;
  auto full = [&](uint32_t s) { return bars + 8u * s; };
  auto empty = [&](uint32_t s) { return bars + 8u * (R + s); };
  const uint32_t b2 = bars + 8u * 2 * R;
  auto pfull = [&](int s) { return b2 + 8u * s; };
  auto pfree = [&](int s) { return b2 + 8u * (kPieceQ + s); };
  const uint32_t b3 = b2 + 8u * 2 * kPieceQ;
  auto k_full = [&](uint32_t i) { return b3 + 8u * i; };
  auto s_full = [&](uint32_t i) { return b3 + 8u * (2 + i); };
  auto s_free = [&](uint32_t i) { return b3 + 8u * (6 + i); };
  auto p_full = [&](uint32_t i) { return b3 + 8u * (10 + i); };
  auto v_full = [&](uint32_t i) { return b3 + 8u * (12 + i); };
  auto pv_done = [&](uint32_t i) { return b3 + 8u * (14 + i); };
  const uint32_t b4 = b3 + 8u * 16;
  auto q_landed = [&](int i) { return b4 + 8u * i; };
  auto q_free = [&](int i) { return b4 + 8u * (2 + i); };
  auto q_full = [&](int i) { return b4 + 8u * (4 + i); };
  const uint32_t drain = b4 + 8u * 8;
  const int4* desc = reinterpret_cast<const int4*>(smem + C::kOffDesc);
  float* fl = reinterpret_cast<float*>(smem + C::kOffFloat);
  float* s_qfac = fl + 64 * 8;  // [4][64] of log2 of a score, by row of q
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc);
  volatile int* s_bad = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::kOffMisc + 16);
  int32_t* warp_tot = reinterpret_cast<int32_t*>(smem + C::kOffMisc + 128);
  int32_t* cu = reinterpret_cast<int32_t*>(smem + C::kOffPlan);

  const int lane = threadIdx.x & 31, tid = threadIdx.x;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int B = p.num_seqs, T = p.q_len;
  const uint32_t H = (uint32_t)p.num_kv_heads;
  const unsigned long long lim = p.timeout_ns, book_ns = p.timeout_ns * kBookkeepingWaits;

  if (tid == 0) {
    for (int s = 0; s < R; ++s) {
      mbar_init(full(s), 2);      // K and V
      mbar_init(empty(s), 2 + 4);  // the warps of the tile's K, those of V
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(s_full(s), 1);
      mbar_init(s_free(s), 8);
    }
    for (int s = 0; s < kPieceQ; ++s) {
      mbar_init(pfull(s), 1);
      mbar_init(pfree(s), kPieceReaders);
      mbar_init(q_full(s), 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full(i), 128);
      mbar_init(p_full(i), 256);
      mbar_init(v_full(i), 256);
      mbar_init(pv_done(i), 1);
      mbar_init(q_landed(i), 1);
      mbar_init(q_free(i), 1);
    }
    mbar_init(drain, 1);
    mbar_init(drain + 8, 1);
    *abort_flag = 0;
    *s_bad = 0;
    cu[0] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kScoreWarp) {
    tc05::tmem_alloc(smem_u32(s_tmem), kTmemCols);
    tc05::tmem_relinquish();
  }
  // rows of q's operand that no query row fills stay 0
  for (uint32_t i = tid; i < 2 * C::kQBuf / 16; i += kThreads)
    reinterpret_cast<uint4*>(smem + C::kOffQ)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (tid < 4 * 64) s_qfac[tid] = 0.f;
  tc05::fence_async_shared();
  tc05::tc_fence_before();
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();
  tc05::tc_fence_after();
  plan_step<kPairCost>(p, cu, s_bad, warp_tot, kThreads, warp == kProducerWarp);
  const uint32_t tmem = *s_tmem;

  // Every role walks the pieces: piece(j) waits for descriptor j and returns whether there is
  // one; the reader hands it back.
  struct Desc {
    int b, h, t0, n, flags, slot, len;
    uint32_t g0;
  };
  auto hand_back = [&](int j) {
    __syncwarp();
    if (lane == 0) mbar_arrive(pfree(j % kPieceQ));
  };
  auto piece = [&](int j, Desc& d, bool back = true) -> bool {
    const int s = j % kPieceQ;
    const bool ok = wait_phase(pfull(s), (j / kPieceQ) & 1u, abort_flag, p.err, book_ns);
    if (!__all_sync(0xffffffffu, ok)) return false;
    const int4 x = desc[2 * s], y = desc[2 * s + 1];
    // (broadcast, so that the compiler keeps what follows from them in uniform registers)
    auto uni = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    d.b = uni(x.x); d.h = uni(x.y); d.t0 = uni(x.z); d.n = uni(x.w);
    d.flags = uni(y.x); d.slot = uni(y.y); d.g0 = (uint32_t)uni(y.z); d.len = uni(y.w);
    if (back) hand_back(j);
    return !(d.flags & kFlagEnd);
  };
  auto wait = [&](uint32_t bar, uint32_t parity) -> bool {  // a warp together
    return __all_sync(0xffffffffu, wait_phase(bar, parity & 1u, abort_flag, p.err, lim));
  };
  // Two barriers (the second only if `also`), half of the lanes at each: one latency where both
  // phases are there already. (A sleeping wait for one after the other was slower, see above.)
  // A lane's own wait acquires only the phase that it looked at, and a vote orders no memory. The
  // warp barrier does, and what is released, acquired and passed through a barrier is ordered for
  // every lane behind it: the arrivals' writes, and a bulk copy's or an MMA's results, whose
  // completion is followed by the proxy fence before it arrives. (What MMAs read or wrote needs
  // tc_fence_after besides, as after any wait.)
  auto wait2 = [&](uint32_t a, uint32_t pa, uint32_t b, uint32_t pb, bool also) -> bool {
    const bool second = also && (lane & 1);
    const bool ok = wait(second ? b : a, second ? pb : pa);
    __syncwarp();
    return ok;
  };

  if (warp >= kProducerWarp) {
    regs_dec<C::kRegsOther>();
    if (warp == kProducerWarp) {
      // ---------------------------------------------------------- producer
      const PartPlan M = part_plan<kMinPart>(p, cu, s_bad);
      UnitCopies<R, C::kBatch> copies;
      copies.ring = base + C::kOffRing;
      copies.full = full(0);
      copies.empty = empty(0);
      copies.policy = evict_first_policy();
      copies.abort_flag = abort_flag;
      copies.stop = p.withhold_copies != 0;  // failure-path test: no copy is issued
      bool lost = false;
      int j = 0;
      if (blockIdx.x == 0 && lane == 0) {
        if (*s_bad) atomicOr(p.err, HPC_DEVCHK_BAD_LENGTH);
        p.owners[0] = (int32_t)M.P;
      }
      auto publish = [&](const Piece& x) {
        const int s = j % kPieceQ;
        const bool end = (x.flags & kFlagEnd) != 0;
        if (lane == 0 && !lost) {
          if (!wait_phase(pfree(s), ((j / kPieceQ) & 1u) ^ 1u, abort_flag, p.err, book_ns)) {
            lost = true;
          } else {
            int4* d = const_cast<int4*>(desc) + 2 * s;
            d[0] = make_int4(x.b, x.h, x.t0, x.n);
            d[1] = make_int4(x.flags, x.slot, (int)copies.g, end ? 0 : __ldg(p.seq_lens + x.b));
            mbar_arrive(pfull(s));  // release: the descriptor is visible to its waiters
          }
        }
        lost = __shfl_sync(0xffffffffu, (int)lost, 0) != 0;
        ++j;
      };
      if (blockIdx.x < M.P) {
        const int4 begun = walk_part<kPairCost>(
            M, cu, B, H, (int)blockIdx.x, [&](const Piece& x) { copies.ahead(p, x); },
            [&](const Piece& x) {
              publish(x);
              copies.copy(p, x);
            });
        if (lane == 0) *reinterpret_cast<int4*>(p.owners + 4 + 4 * blockIdx.x) = begun;
      }
      publish(Piece{0, 0, 0, 0, kFlagEnd, -1});
      named_bar_sync(3, kThreads);
      if (*abort_flag) copies.drain(p);
      return;
    }
    if (warp == kScoreWarp || warp == kValueWarp) {
      // ------------------------------------------------------- MMA issue
      // A warp for each product; it runs the whole schedule, one elected lane issues. Two,
      // since waits and issue are a serial chain of about 600 clk a step for each: a wait
      // takes 100 clk even when the phase is there already.
      const bool leader = tc05::elect_one() != 0;
      bool ok = true, any = false;
      uint32_t step = 0;
      Desc d;
      if (warp == kScoreWarp) {
        constexpr uint32_t kIdS = tc05::idesc_f16_f32(128, COLS, false, false);
        const uint64_t qd = tc05::smem_desc_sw128(base + C::kOffQ, 16, 1024);
        for (int j = 0; ok && piece(j, d); ++j) {
          const int steps = (d.n + 1) / 2;
          ok = wait(q_full(j & 3), j >> 2);
          for (int k = 0; ok && k < steps; ++k, ++step) {
            const uint32_t i = step & 1, s4 = step & 3;
            // K, and the scores of four steps before read
            ok = wait2(k_full(i), step >> 1, s_free(s4), (step >> 2) - 1, step >= 4);
            if (!ok) break;
            tc05::tc_fence_after();
            if (leader) {
              const uint32_t sd = tmem + kColS + 64u * s4, a = tmem + kColK + 64u * i;
              const uint64_t b = qd + (uint64_t)((j & 1) * (C::kQBuf >> 4));
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                tc05::mma_f16_ts(sd, a + 8 * kk, b + (kk >> 2) * (C::kQHalf >> 4) + (kk & 3) * 2,
                                 kIdS, kk > 0 ? 1u : 0u);
              tc05::mma_commit(s_full(s4));
              if (k == steps - 1) tc05::mma_commit(q_free(j & 1));
            }
            __syncwarp();
            any = true;
          }
        }
      } else {
        constexpr uint32_t kIdO = tc05::idesc_f16_f32(128, COLS, true, true);
        const uint64_t vd = tc05::smem_desc_sw128(base + C::kOffV, kVTile / 2, 1024);
        const uint64_t pd = tc05::smem_desc_sw128(base + C::kOffP, 16, 1024);
        for (int j = 0; ok && piece(j, d); ++j) {
          const int steps = (d.n + 1) / 2;
          for (int k = 0; ok && k < steps; ++k, ++step) {
            const uint32_t i = step & 1;
            // (that O^T's rows of the piece before were written out follows from P^T)
            ok = wait2(p_full(i), step >> 1, v_full(i), step >> 1, true);
            if (!ok) break;
            tc05::tc_fence_after();
            if (leader) {
              const uint64_t a = vd + (uint64_t)(i * (2 * kVTile >> 4));
              const uint64_t b = pd + (uint64_t)(i * (kPBuf >> 4));
#pragma unroll
              for (int kk = 0; kk < 8; ++kk) {
                if (kk == 4 && 2 * k + 1 == d.n) break;
                tc05::mma_f16_ss(tmem + kColO,
                                 a + (kk >> 2) * (kVTile >> 4) + (kk & 3) * (2048 >> 4),
                                 b + kk * (2048 >> 4), kIdO, k == 0 && kk == 0 ? 0u : 1u);
              }
              tc05::mma_commit(pv_done(i));
            }
            __syncwarp();
            any = true;
          }
        }
      }
      if (leader && any) {
        const uint32_t mine = drain + (warp == kScoreWarp ? 0 : 8);
        tc05::mma_commit(mine);  // every MMA this lane issued has completed
        wait_phase(mine, 0, abort_flag, p.err, 1000000000ull, false);
      }
      __syncwarp();
      tc05::tc_fence_before();
      named_bar_sync(3, kThreads);
      if (warp == kScoreWarp) {
        tc05::tc_fence_after();
        tc05::tmem_dealloc(tmem, kTmemCols);
      }
      return;
    }
    // ------------------------------------------------------ copies of q
    Desc d = {};
    int q_pieces = 0;
    for (int j = 0; piece(j, d); ++j) {
      const int i = j & 1;
      // once the MMAs on the buffer's previous rows are done
      if (j >= 2 && !wait(q_free(i), (j >> 1) - 1)) break;
      if (p.withhold_copies) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(q_landed(i), (uint32_t)(T * kGroup * kHeadDim * 2));
        const uint32_t dq = base + C::kOffQ + i * C::kQBuf;
        tc05::tma_load_4d(dq, &tmq, q_landed(i), 0, d.h * kGroup, 0, d.b);
        tc05::tma_load_4d(dq + C::kQHalf, &tmq, q_landed(i), 64, d.h * kGroup, 0, d.b);
      }
      q_pieces = j + 1;
    }
    // (rows that nobody waited for may still be landing)
    for (int j = q_pieces > 2 ? q_pieces - 2 : 0; *abort_flag && lane == 0 && j < q_pieces; ++j)
      wait_phase(q_landed(j & 1), (j >> 1) & 1u, abort_flag, p.err, 1000000000ull, false);
    __syncwarp();  // (lane 0 alone may have waited; the barrier is the whole warp's)
    named_bar_sync(3, kThreads);
    return;
  }

  if (warp >= kVWarp0) {
    regs_dec<C::kRegsV>();
    // ------------------------------------------------------ V to f16
    // Sixteen elements of a token to a thread: eight bytes of codes times their scale, into
    // the two 64-element halves of the tile, 128-byte swizzle. Shared memory's bandwidth is
    // what this kernel has least of, so no access here meets another's bank: an 8-byte load is
    // served 16 threads at a time, two rows that lie 8 apart (8 rows of 18 words move 16
    // banks); a 16-byte store 8 at a time, one row of which the upper half's threads store
    // their second eight elements first. Rows past the sequence become 0, whatever the slots
    // hold.
    const int tile = (warp - kVWarp0) >> 2;  // of the step's two
    const int ct = tid & 127;
    const int c = ct & 7, up = c >> 2;
    const int r0 = ((ct >> 3) & 1) * 8 + (ct >> 5) * 2 + ((ct >> 4) & 1);
    uint32_t step = 0;
    Desc d;
    bool ok = true;
    for (int j = 0; ok && piece(j, d); ++j) {
      for (int k = tile; ok && k < d.n + tile; k += 2, ++step) {
        const uint32_t i = step & 1, u = d.g0 + k, slot = u % R;
        const bool there = k < d.n;
        // the copy, and the products of two steps before (for a step's missing second tile too:
        // an arrival counts for the barrier's current phase)
        ok = there ? wait2(full(slot), u / R, pv_done(i), (step >> 1) - 1, step >= 2)
                   : step < 2 || wait(pv_done(i), (step >> 1) - 1);
        if (!ok) break;
        if (!there) {
          mbar_arrive(v_full(i));
          continue;
        }
        const uint32_t src = base + C::kOffRing + slot * (2 * kKv4Tile) + kKv4Tile;
        const uint32_t dst =
            base + C::kOffV + (i * 2 + tile) * kVTile + (c >> 2) * (kVTile / 2);
        const int stored = d.len - (d.t0 + k) * kBlockTokens;
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          const int t = it * 16 + r0;
          const uint32_t row = src + t * kKv4Row;
          const uint2 x = *reinterpret_cast<const uint2*>(__cvta_shared_to_generic(row + 8 * c));
          uint32_t f = *reinterpret_cast<const uint8_t*>(__cvta_shared_to_generic(row + kKv4Codes + c));
          if (t >= stored) f = 0;
          f = both_low(kv4_scales(f));
          uint32_t w[2][4];
          e2m1x8_to_f16(up ? x.y : x.x, w[0]);
          e2m1x8_to_f16(up ? x.x : x.y, w[1]);
          const int cc = (c & 3) * 2;
          const uint32_t to = dst + t * 128;
#pragma unroll
          for (int y = 0; y < 2; ++y) {
#pragma unroll
            for (int z = 0; z < 4; ++z) w[y][z] = mul_f16x2(w[y][z], f);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             to + ((uint32_t)((cc + (y ^ up)) ^ (t & 7)) << 4)),
                         "r"(w[y][0]), "r"(w[y][1]), "r"(w[y][2]), "r"(w[y][3])
                         : "memory");
          }
        }
        tc05::fence_async_shared();  // the MMAs read the tile through the async proxy
        mbar_arrive(v_full(i));
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(slot));
      }
    }
    named_bar_sync(3, kThreads);
    return;
  }

  if (warp >= kKWarp0) {
    regs_dec<C::kRegsK>();
    // ------------------------ q to f16; K to f16, in tensor memory
    // A thread is a token of the step, its lane of tensor memory.
    const int row = tid - 32 * kKWarp0, tile = row >> 6;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    uint32_t step = 0;
    Desc d;
    bool ok = true;
    for (int j = 0; ok && piece(j, d); ++j) {
      // The piece's query rows, in place: eight threads a row, 16 bytes of each half to a
      // thread in the order in which they lie (below the swizzle). A power of two of the row's
      // own puts its largest element in [2^14, 2^15).
      if (!(ok = wait(q_landed(j & 1), j >> 1))) break;
#pragma unroll
      for (int r = row >> 3; r < T * kGroup; r += 16) {
        uint4* at = reinterpret_cast<uint4*>(smem + C::kOffQ + (j & 1) * C::kQBuf) + r * 8 + (row & 7);
        uint4 w[2] = {at[0], at[C::kQHalf / 16]};
        uint32_t big = 0;  // the largest bf16 without its sign, as an integer
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t x[4] = {w[y].x, w[y].y, w[y].z, w[y].w};
#pragma unroll
          for (int z = 0; z < 4; ++z) big = max(big, max(x[z] & 0x7FFF0000u, (x[z] & 0x7FFFu) << 16));
        }
        const uint32_t eight = 0xFFu << (lane & 24);
        big = __reduce_max_sync(eight, big);
        int e = 0;
        if (big > 0) {
          e = 14 - ((int)(big >> 23) - 127);
          e = e < -113 ? -113 : (e > 100 ? 100 : e);
        }
        const float sc = __uint_as_float((uint32_t)(e + 127) << 23);
        auto scaled = [&](uint32_t x) {
          return pack_f16(__uint_as_float(x << 16) * sc, __uint_as_float(x & 0xFFFF0000u) * sc);
        };
#pragma unroll
        for (int y = 0; y < 2; ++y)
          at[y * (C::kQHalf / 16)] = make_uint4(scaled(w[y].x), scaled(w[y].y), scaled(w[y].z), scaled(w[y].w));
        // A factor of 0 would make NaN of masked scores, an infinite one of scores of 0. Four
        // sets of factors and barriers, as descriptors: the softmax may be behind by that many
        // pieces.
        if ((row & 7) == 0)
          s_qfac[(j & 3) * 64 + r] = fminf(
              fmaxf(p.score_scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23), FLT_MIN), FLT_MAX);
      }
      tc05::fence_async_shared();  // the MMAs read q through the async proxy
      mbar_arrive(q_full(j & 3));
      const int steps = (d.n + 1) / 2;
      for (int k = 0; ok && k < steps; ++k, ++step) {
        const uint32_t i = step & 1, u = d.g0 + 2 * k + tile, slot = u % R;
        const bool there = 2 * k + tile < d.n;
        // the copy, and the scores of two steps before
        const uint32_t before = s_full((step - 2) & 3);
        ok = there ? wait2(full(slot), u / R, before, (step - 2) >> 2, step >= 2)
                   : step < 2 || wait(before, (step - 2) >> 2);
        if (!ok) break;
        if (there) {
          tc05::tc_fence_after();
          const uint32_t src = base + C::kOffRing + slot * (2 * kKv4Tile) + (row & 63) * kKv4Row;
          auto load = [&](int x) {
            return *reinterpret_cast<const uint2*>(__cvta_shared_to_generic(src + 8 * x));
          };
          const uint2 sc = load(8);
          // (unrolled it is faster only beside 48 rows: 109.6 us for 112.2 with 6 tokens, but
          // 100.7 for 98.6 with 4 and 127.3 for 126.4 with 8)
#pragma unroll(COLS == 48 ? 2 : 1)
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t w[32];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint2 c = load(4 * hf + x);
              const uint32_t pair = kv4_scales((hf ? sc.y : sc.x) >> (16 * (x >> 1)));
              const uint32_t f = x & 1 ? both_high(pair) : both_low(pair);
              uint32_t a[4], b[4];
              e2m1x8_to_f16(c.x, a);
              e2m1x8_to_f16(c.y, b);
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                w[8 * x + y] = mul_f16x2(a[y], f);
                w[8 * x + 4 + y] = mul_f16x2(b[y], f);
              }
            }
            tc05::tmem_st32(tmem + kColK + 64u * i + 32u * hf + lanes, w);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(empty(slot));  // (the row has been read)
          tc05::tmem_wait_st();
          tc05::tc_fence_before();
        }
        mbar_arrive(k_full(i));
      }
    }
    named_bar_sync(3, kThreads);
    return;
  }

  regs_inc<C::kRegsSoftmax>();
  // ------------------------------------------------- softmax, pieces' ends
  // Two groups of four warps share the query rows. The warps of a group take every way out
  // together: barriers lie between.
  constexpr int N = C::kHalf;
  const int grp = warp >> 2, c0 = grp * N;  // this group's rows: c0 .. c0 + N - 1
  const int row = tid & 127;                // token of the step, element d of the head
  const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
  const uint32_t od = tmem + kColO + lanes + c0;
  const int bar = 6 + grp;
  float* s_true = fl + c0;        // references: the largest score so far, or -inf
  float* s_ref = fl + 64 + c0;    // what is subtracted: the same, 0 for -inf
  float* s_alpha = fl + 128 + c0;
  float* s_inv = fl + 192 + c0;
  float* s_part = fl + 256 + c0;  // [4][64]
  uint32_t step = 0;
  Desc d = {};
  for (int j = 0;; ++j) {
    bool ok = piece(j, d, false);
    if (ok) ok = wait(q_full(j & 3), j >> 2);
    if (any_of(bar, 128, !ok)) break;
    const int steps = (d.n + 1) / 2;
    const float* fac = s_qfac + (j & 3) * 64 + c0;
    // References and factors stay in registers: a 16-byte broadcast takes shared memory four
    // cycles, as any 512 bytes do (6 tokens 130 -> 113 us, 8 153 -> 131).
    float ref[N] = {}, factor[N];
#pragma unroll
    for (int c = 0; c < N; ++c) factor[c] = fac[c];
    float l[N];
#pragma unroll
    for (int c = 0; c < N; ++c) l[c] = 0.f;
    const int end = (d.t0 + d.n) * kBlockTokens < d.len ? (d.t0 + d.n) * kBlockTokens : d.len;
    for (int k = 0; k < steps; ++k, ++step) {
      const uint32_t i = step & 1;
      // the scores; P^T's buffer free after the products of two steps before
      ok = wait2(s_full(step & 3), step >> 2, pv_done(i), (step >> 1) - 1, step >= 2);
      tc05::tc_fence_after();
      const int at = (d.t0 + 2 * k) * kBlockTokens, pos = at + row;
      float s[N];
      auto scores = [&] {
        const uint32_t sd = tmem + kColS + 64u * (step & 3) + lanes + c0;
#pragma unroll
        for (int c = 0; c < N; c += 8) tmem_ld8(sd + c, s + c);
        tc05::tmem_wait_ld();
        if (at + 128 > end || at + 128 > d.len - (T - 1)) {  // some see less than all 128
#pragma unroll
          for (int t = 0; t < N / 8; ++t) {
            const int mine = d.len - (T - 1 - (c0 / 8 + t));  // (of rows that no token fills: any)
            if (pos >= mine || pos >= end) {
#pragma unroll
              for (int c = 0; c < 8; ++c) s[8 * t + c] = -INFINITY;
            }
          }
        }
      };
      // (a product and a difference, not one FMA: the largest product has to give exactly 0,
      // and what rounding took from a reference of 2^30 is no small number)
      auto less_reference = [&] {
#pragma unroll
        for (int c = 0; c < N; ++c) s[c] = __fsub_rn(__fmul_rn(s[c], factor[c]), ref[c]);
      };
      scores();
      bool passed = k == 0;
      if (!passed) {
        float over[2] = {-INFINITY, -INFINITY};
        less_reference();
#pragma unroll
        for (int c = 0; c < N; ++c) over[c & 1] = fmaxf(over[c & 1], s[c]);
        passed = fmaxf(over[0], over[1]) > kPassed;
      }
      if (any_of(bar, 128, passed || !ok)) {
        if (any_of(bar, 128, !ok)) {
          ok = false;
          break;
        }
        // references: the rows' maxima over the step, of each warp and then of all
        if (k > 0) scores();
        reduce_rows<true, 16, N>(s, 0, s_part + (warp & 3) * 64, lane);
        named_bar_sync(bar, 128);
        if (row < N) {
          const float old = k == 0 ? -INFINITY : s_true[row];
          const float mx = fmaxf(fmaxf(s_part[row], s_part[64 + row]),
                                 fmaxf(s_part[128 + row], s_part[192 + row])) * fac[row];
          const float now = fmaxf(old, mx);
          s_true[row] = now;
          s_ref[row] = now == -INFINITY ? 0.f : now;
          s_alpha[row] = now == -INFINITY ? 1.f : ex2(old - now);
        }
        named_bar_sync(bar, 128);
#pragma unroll
        for (int c = 0; c < N; ++c) ref[c] = s_ref[c];
        if (k > 0) {
          // O is stable once the products of the step before are done
          ok = wait(pv_done(i ^ 1), (step - 1) >> 1);
          if (any_of(bar, 128, !ok)) {
            ok = false;
            break;
          }
          tc05::tc_fence_after();
#pragma unroll
          for (int c = 0; c < N; c += 8) {
            float o[8];
            tmem_ld8(od + c, o);
            tc05::tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 8; ++x) o[x] *= s_alpha[c + x];
            tmem_st8(od + c, o);
          }
          tc05::tmem_wait_st();
#pragma unroll
          for (int c = 0; c < N; ++c) l[c] *= s_alpha[c];
        }
        scores();
        less_reference();
      }
      const uint32_t prow = base + C::kOffP + i * kPBuf + row * 128;
#pragma unroll
      for (int c = 0; c < N; c += 8) {
        float e[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          e[x] = ex2(s[c + x]);
          l[c + x] += e[x];
        }
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                         prow + ((uint32_t)(((c0 + c) >> 3) ^ (row & 7)) << 4)),
                     "r"(pack_f16(e[0], e[1])), "r"(pack_f16(e[2], e[3])),
                     "r"(pack_f16(e[4], e[5])), "r"(pack_f16(e[6], e[7]))
                     : "memory");
      }
      tc05::fence_async_shared();
      tc05::tc_fence_before();  // (O was rescaled before the products that this allows)
      mbar_arrive(p_full(i));
      __syncwarp();
      if (lane == 0) mbar_arrive(s_free(step & 3));
    }
    hand_back(j);     // (q's factors were read until here)
    if (!ok) break;  // (of all, see above)
    // ---- the piece's end: sums over the tokens (each lane ends with some of the rows)
    reduce_rows<false, 16, N>(l, 0, s_part + (warp & 3) * 64, lane);
    named_bar_sync(bar, 128);
    const int mine = c0 + row;  // a query row
    if (row < N && mine < T * kGroup) {
      const float sum = (s_part[row] + s_part[64 + row]) + (s_part[128 + row] + s_part[192 + row]);
      const float m = s_true[row];
      s_inv[row] = sum == 0.f ? 0.f : p.v_scale / sum;
      if (!(d.flags & kFlagWhole)) {
        reinterpret_cast<float2*>(p.ws_ml)[(int64_t)d.slot * T * kGroup + mine] = make_float2(m, sum);
      } else if (p.lse) {
        p.lse[(int64_t)d.b * p.l_sb + (int64_t)(mine / kGroup) * p.l_st +
              (int64_t)(d.h * kGroup + mine % kGroup) * p.l_sh] =
            sum == 0.f ? -INFINITY : (m + __log2f(sum)) * kLn2;
      }
    }
    named_bar_sync(bar, 128);
    ok = wait(pv_done((step - 1) & 1), (step - 1) >> 1);
    if (any_of(bar, 128, !ok)) break;
    tc05::tc_fence_after();
#pragma unroll
    for (int x8 = 0; x8 < N / 8; ++x8) {
      const int t = c0 / 8 + x8;
      if (t >= T) break;
      float o[8];
      tmem_ld8(od + 8 * x8, o);
      tc05::tmem_wait_ld();
      if (d.flags & kFlagWhole) {
        __nv_bfloat16* out = p.out + (int64_t)d.b * p.o_sb + (int64_t)t * p.o_st +
                             (int64_t)(d.h * kGroup) * p.o_sh + row;
#pragma unroll
        for (int x = 0; x < 8; ++x)
          out[x * p.o_sh] = __float2bfloat16_rn(o[x] * s_inv[8 * x8 + x]);
      } else {
        float* ws = reinterpret_cast<float*>(p.ws) +
                    ((int64_t)d.slot * T + t) * (kGroup * kHeadDim) + row;
#pragma unroll
        for (int x = 0; x < 8; ++x) ws[x * kHeadDim] = o[x];
      }
    }
    tc05::tc_fence_before();  // (before the next piece's P^T, which lets O^T be written again)
  }
  // sequences without tiles (or a step that cannot be): out = 0, lse = -inf
  if (d.flags & kFlagEnd) {
    for (int b = (int)blockIdx.x * 8 + warp; b < B; b += (int)gridDim.x * 8) {
      if (!*s_bad && cu[b + 1] != cu[b]) continue;
      for (int t = 0; t < T; ++t)
        for (int x = lane; x < (int)H * kGroup; x += 32) {
          uint4* o = reinterpret_cast<uint4*>(p.out + (int64_t)b * p.o_sb + (int64_t)t * p.o_st +
                                              (int64_t)x * p.o_sh);
#pragma unroll
          for (int i = 0; i < kHeadDim / 8; ++i) o[i] = make_uint4(0u, 0u, 0u, 0u);
          if (p.lse)
            p.lse[(int64_t)b * p.l_sb + (int64_t)t * p.l_st + (int64_t)x * p.l_sh] = -INFINITY;
        }
    }
  }
  tc05::tc_fence_before();
  named_bar_sync(3, kThreads);
}

template <int COLS>
cudaError_t launch_cols(const Kv4DecodeParams& p, const CUtensorMap& tq, int grid, cudaStream_t stream) {
  using C = Cfg<COLS>;
  auto kern = kv4_tc_kernel<COLS>;
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = once_per_device(configured, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)C::kSmemBytesMax);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes + 4 * ((size_t)p.num_seqs + 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p, tq);
}

}  // namespace

cudaError_t launch_kv4_tc(const Kv4DecodeParams& p, const CUtensorMap& tq, int grid,
                          cudaStream_t stream) {
  if (p.num_seqs > kKv4MaxSeqs) return cudaErrorInvalidValue;
  if (p.q_len <= 2) return launch_cols<16>(p, tq, grid, stream);
  if (p.q_len <= 4) return launch_cols<32>(p, tq, grid, stream);
  if (p.q_len <= 6) return launch_cols<48>(p, tq, grid, stream);
  return launch_cols<64>(p, tq, grid, stream);
}

}  // namespace hpc
