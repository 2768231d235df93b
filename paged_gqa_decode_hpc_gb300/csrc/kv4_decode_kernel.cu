// Decode attention of one new token per sequence over a 4-bit paged cache: planned, computed
// and merged by a single persistent kernel. (Several tokens: kv4_tc_kernel.cu.)
//
//   s_t = scale * q . k_t,  out = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m)
//
// over a sequence's 64-token tiles, one (tile, KV head) unit after another with a
// running maximum and sum; the 8 query heads of a KV head share a unit's K and V in
// registers. The plan (kv4_plan.cuh) gives every CTA an equal part of the units, taken in
// pieces of one (sequence, KV head) pair, whose states are joined by log-sum-exp.
//
// What bounds it: the consumer warps' own latencies; nothing that they share is full. A unit is
// 9216 bytes, 206 ns of an SM's share of 6.8 TB/s (390 cycles), in which its 16384 codes have to
// become f16 operands: about 1080 warp instructions, 64 of them MMAs, 270 issue cycles of the
// SM. So a warp takes a unit by itself, and no value moves between warps. Measured: 31 sequences
// of 4096 and one of 131072 positions of 8 KV heads 55.9 us (298 MB, 5.3 TB/s); while its SMs are
// active they issue in 52 % of the cycles, and no pipe is busier than the ALU (47 %; FMA 31 %,
// tensor 25 %): two consumer warps to a scheduler, and a warp goes 7.7 cycles between two
// instructions. 64 sequences of 200 to 6000 30.2 us, of which 5 are the plan, the first unit's
// two dependent loads and the last states' way to memory.
//
// How a unit gets into the MMAs (mma.sync m16n8k16, f16; S^T = K Q^T, O^T = V^T P^T):
//  * A tile is copied as it lies in memory, 64 rows of 72 bytes. Rows are 18 words
//    apart, so rows 4i + s, i = 0..7 (s fixed) start 8 banks apart modulo 32, and four
//    of them with eight bytes of four lanes each cover all banks once.
//  * The MMAs do not care in which order tokens, or the elements of a head, come, as
//    long as both operands agree. Row i of an 8-row group s of a 32-token half is
//    token 4 I(i) + s with I = 0 6 1 7 2 4 3 5: rows 0..3 and 4..7, which one access of K
//    takes together, and rows 0 2 4 6 and 1 3 5 7, which one access of V does, then lie
//    in different banks.
//  * K: lane (g, c) reads eight bytes, elements 16c .. 16c + 15 and 64 + 16c .. , of its
//    rows: neighbouring codes are neighbours of the contraction, and a conversion of a
//    byte gives a register of the operand. Two scales a row.
//  * V: its contraction runs over tokens, whose codes lie 72 bytes apart. Lane (g, c)
//    reads eight bytes, elements 16g .. 16g + 15, of two tokens, and two shifts and two
//    bit selects make bytes of one element's codes of both tokens. One scale a token.
//  * Codes times scales are exact in f16 (kv4.cuh). Each row of Q takes a power of two that puts
//    its largest element in [2^14, 2^15), P is rounded to f16 (2^-11), sums and states
//    are fp32. The row maximum moves only when a score passes it by 8 (in log2 units),
//    so that most units neither reduce it over the lanes nor rescale the sums; P then
//    stays below 2^8.
//  * Slots past a sequence's end may hold anything: scores of theirs are masked after
//    the product, and V's scales of theirs become 0 (codes are finite).
#include <cfloat>

#include "decode_common.cuh"
#include "hpc_internal.h"
#include "kv4.cuh"
#include "kv4.h"
#include "kv4_plan.cuh"
#include "kv4_state.cuh"
#include "ptx.cuh"

namespace hpc {
namespace {

// Warpgroups 0 and 1: consumer warps. Warpgroup 2: epilogue, each of its warps a quarter of
// every state. Warpgroup 3: the producer warp and three that leave at once.
constexpr int kConsumerWarps = 8, kEpilogueWarp0 = 8, kEpilogueWarps = 4, kProducerWarp = 12;
// Units that a pair counts for beside its own, and that a CTA is worth starting for (64
// sequences of 200 to 6000 positions 32.9 us with 2, 29.7 with 4, 30.2 with 6; 8 short ones 9.4
// us with parts of at least 8 units, 7.9 with 4).
constexpr int kPairCost = 4, kMinPart = 4;
constexpr int kThreads = 512;
constexpr int kPieceQ = 4;                        // piece descriptors in flight
constexpr int kDescInts = 8;
constexpr int kDepVec = 5;                        // 16-byte words per lane of a deposited state
constexpr int kStage = 2 * kKv4Tile;
constexpr int kQRow = kHeadDim * 2;               // bytes of a row of q in shared memory
constexpr int kFan = 16;                          // pieces of a pair that are joined at once

struct Cfg {
  static constexpr int kGroups = kConsumerWarps;  // units in work at once, each warp's in its own slots
  static constexpr int kBufs = 2;                 // deposit buffers: warps may run a piece ahead
  static constexpr int kDepBytes = kConsumerWarps * kDepVec * 32 * 16;
  static constexpr int kQBytes = kGroup * kQRow;  // a piece's rows of q
  static constexpr int kFixed =
      kBufs * kDepBytes + kPieceQ * kQBytes + 1024 /* barriers, descriptors, scan */ + 128 + 4 * (kKv4MaxSeqs + 1);
  static constexpr int kStages = (227 * 1024 - kFixed) / kStage / kGroups * kGroups;
  static constexpr int kBatch = kStages < 16 ? 8 : 16;  // units that the producer takes at once
  static constexpr int kDepOff = kStages * kStage;
  static constexpr int kQOff = kDepOff + kBufs * kDepBytes;
  static constexpr int kBarOff = kQOff + kPieceQ * kQBytes;
  // full, empty, piece full, piece free, deposit full, deposit free
  static constexpr int kNumBars = 2 * kStages + 2 * kPieceQ + 2 * kBufs;
  static constexpr int kDescOff = kBarOff + 8 * ((kNumBars + 1) / 2 * 2);
  static constexpr int kMiscOff = kDescOff + 4 * kDescInts * kPieceQ;
  static constexpr int kPlanOff = kMiscOff + 256;  // abort flag, flags, scan scratch
  static constexpr int kSmemBytes = 128 /* alignment slack */ + kPlanOff;
  static constexpr int kSmemBytesMax = kSmemBytes + 4 * (kKv4MaxSeqs + 1);
  static_assert(kSmemBytesMax <= 227 * 1024, "shared memory");
  static_assert(kBatch <= kStages, "a slot to each unit of a batch");
  // Registers a thread, of the 128 that the launch gives each (one warp of each warpgroup
  // to an SM sub-partition, so that the four add up to 512).
  static constexpr int kRegsConsumer = 168;
  static constexpr int kRegsEpilogue = 104;
  static constexpr int kRegsProducer = 72;
  static_assert(2 * kRegsConsumer + kRegsEpilogue + kRegsProducer == 512, "registers");
};
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  return *reinterpret_cast<const uint2*>(__cvta_shared_to_generic(a));
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
  return *reinterpret_cast<const uint8_t*>(__cvta_shared_to_generic(a));
}
__device__ __forceinline__ uint32_t prmt2(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
// (a & m) | (b & ~m)
__device__ __forceinline__ uint32_t select_bits(uint32_t a, uint32_t b, uint32_t m) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xE2;" : "=r"(r) : "r"(a), "r"(m), "r"(b));
  return r;
}

// The token of row i of group 0 of a half, over 4.
__device__ __forceinline__ int row_token(int i) { return (int)((0x53427160u >> (4 * i)) & 7u); }

// 8 rows of q in shared memory as B operands in K's order of elements:
// register j of k-step ks holds elements 64 (ks / 4) + 16 c + 4 (ks % 4) + 2 j, + 1 of query
// head g. Each row takes a power of two of its own, so that no head's size (or infinity)
// costs another one bits; inv receives the factors that undo those of this lane's columns of
// the scores, 2c and 2c + 1.
__device__ __forceinline__ void load_q4(uint32_t q, int lane, uint32_t (&qf)[8][2], float (&inv)[2]) {
  const int g = lane >> 2, c = lane & 3;
  const uint32_t row = q + (uint32_t)(g * kQRow + 32 * c);
  uint4 u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u[i].x), "=r"(u[i].y), "=r"(u[i].z), "=r"(u[i].w)
                 : "r"(row + 128 * (i >> 1) + 16 * (i & 1)));
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[e] << 16)),
                               fabsf(__uint_as_float(w[e] & 0xFFFF0000u))));
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  int e = 0;
  if (amax > 0.f) {
    e = 14 - ((int)((__float_as_uint(amax) >> 23) & 0xFF) - 127);
    e = e < -113 ? -113 : (e > 100 ? 100 : e);
  }
  const float sc = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
    for (int x = 0; x < 4; ++x)
      qf[2 * i + (x >> 1)][x & 1] =
          pack_f16(__uint_as_float(w[x] << 16) * sc, __uint_as_float(w[x] & 0xFFFF0000u) * sc);
  }
  const float undo = __uint_as_float((uint32_t)(127 - e) << 23);
  inv[0] = __shfl_sync(0xffffffffu, undo, 8 * c);  // (a lane of row 2c)
  inv[1] = __shfl_sync(0xffffffffu, undo, 8 * c + 4);
}

// One unit, of whose tokens `stored` are in the sequence.
__device__ __forceinline__ void compute_unit4(uint32_t kb, uint32_t vb,
                                              const uint32_t (&qf)[8][2], int stored,
                                              const float (&sl2)[2], float (&m)[2], float (&l)[2], float (&acc)[8][4],
                                              int lane) {
  const int g = lane >> 2, c = lane & 3;
  const int ig = row_token(g);
  float s[4][4];
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) s[mt][0] = s[mt][1] = s[mt][2] = s[mt][3] = 0.f;

  // ---- S^T = K Q^T: rows g and g + 8 of step mt are tokens 32 (mt / 2) + 4 I(g) + 2 (mt % 2) + 0, 1
  const uint32_t k_lane = kb + (uint32_t)(ig * 4 * kKv4Row + 8 * c);
  const uint32_t ks_lane = kb + (uint32_t)(ig * 4 * kKv4Row + kKv4Codes);
  const uint32_t sel = (uint32_t)(c | ((4 + c) << 4));
  uint32_t f0[4], f1[4];
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) {
    const uint32_t off = (uint32_t)((32 * (mt >> 1) + 2 * (mt & 1)) * kKv4Row);
    const uint2 y0 = lds64(ks_lane + off), y1 = lds64(ks_lane + off + kKv4Row);
    f0[mt] = kv4_scales(prmt2(y0.x, y0.y, sel));
    f1[mt] = kv4_scales(prmt2(y1.x, y1.y, sel));
  }
  // (the four steps mt side by side: their chains of MMAs are independent)
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    uint2 x0[4], x1[4];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      const uint32_t off = (uint32_t)((32 * (mt >> 1) + 2 * (mt & 1)) * kKv4Row + 32 * hf);
      x0[mt] = lds64(k_lane + off);
      x1[mt] = lds64(k_lane + off + kKv4Row);
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        const uint32_t g0 = hf ? both_high(f0[mt]) : both_low(f0[mt]);
        const uint32_t g1 = hf ? both_high(f1[mt]) : both_low(f1[mt]);
        uint32_t a[4], b[4];
        e2m1x8_to_f16(w ? x0[mt].y : x0[mt].x, a);
        e2m1x8_to_f16(w ? x1[mt].y : x1[mt].x, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = mul_f16x2(a[i], g0);
          b[i] = mul_f16x2(b[i], g1);
        }
        const int ks = 4 * hf + 2 * w;
        mma_f16(s[mt], a[0], b[0], a[1], b[1], qf[ks][0], qf[ks][1]);
        mma_f16(s[mt], a[2], b[2], a[3], b[3], qf[ks + 1][0], qf[ks + 1][1]);
      }
    }
  }

  // ---- online softmax in the log2 domain; columns 2c and 2c + 1
  uint32_t pb[4][2];
  if (stored < 64) {
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (32 * (mt >> 1) + 4 * ig + 2 * (mt & 1) + r >= stored)
          s[mt][2 * r] = s[mt][2 * r + 1] = -INFINITY;
  }
  float mx0 = fmaxf(s[0][0], s[0][2]), mx1 = fmaxf(s[0][1], s[0][3]);
#pragma unroll
  for (int mt = 1; mt < 4; ++mt) {
    mx0 = fmaxf(mx0, fmaxf(s[mt][0], s[mt][2]));
    mx1 = fmaxf(mx1, fmaxf(s[mt][1], s[mt][3]));
  }
  mx0 *= sl2[0];
  mx1 *= sl2[1];
  if (__any_sync(0xffffffffu, mx0 > m[0] + 8.f || mx1 > m[1] + 8.f)) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
    }
    const float n0 = fmaxf(m[0], mx0), n1 = fmaxf(m[1], mx1);
    const float al0 = n0 == -INFINITY ? 1.f : ex2(m[0] - n0);
    const float al1 = n1 == -INFINITY ? 1.f : ex2(m[1] - n1);
    m[0] = n0;
    m[1] = n1;
    l[0] *= al0;
    l[1] *= al1;
#pragma unroll
    for (int dm = 0; dm < 8; ++dm) {
      acc[dm][0] *= al0;
      acc[dm][1] *= al1;
      acc[dm][2] *= al0;
      acc[dm][3] *= al1;
    }
  }
  // (a row that has seen no position yet: its scores are all -inf, its P is 0)
  // (a product and a difference, not one FMA: the largest product has to give exactly 0, and
  // what rounding took from a maximum of 2^30 is no small number)
  const float r0 = m[0] == -INFINITY ? 0.f : m[0];
  const float r1 = m[1] == -INFINITY ? 0.f : m[1];
  auto less = [&](float x, float f, float r) { return ex2(__fsub_rn(__fmul_rn(x, f), r)); };
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) {
    const float e0 = less(s[mt][0], sl2[0], r0), e1 = less(s[mt][1], sl2[1], r1);
    const float e2 = less(s[mt][2], sl2[0], r0), e3 = less(s[mt][3], sl2[1], r1);
    l[0] += e0 + e2;
    l[1] += e1 + e3;
    pb[mt][0] = movm_trans(pack_f16(e0, e1));
    pb[mt][1] = movm_trans(pack_f16(e2, e3));
  }

  // ---- O^T += V^T P^T: the k pairs of step kt are tokens ta, tb (rows 2c, 2c + 1) and ta + 1, tb + 1
  const int ta = 4 * row_token(2 * c), tb = 4 * row_token(2 * c + 1);
  const uint32_t va_lane = vb + (uint32_t)(ta * kKv4Row), vb_lane = vb + (uint32_t)(tb * kKv4Row);
#pragma unroll
  for (int kt = 0; kt < 4; ++kt) {
    const int tok = 32 * (kt >> 1) + 2 * (kt & 1);
    const uint32_t off = (uint32_t)(tok * kKv4Row);
    uint32_t f[2];
    uint2 xa[2], xb[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint32_t o = off + (uint32_t)(r * kKv4Row);
      xa[r] = lds64(va_lane + o + 8 * g);
      xb[r] = lds64(vb_lane + o + 8 * g);
      f[r] = lds_u8(va_lane + o + kKv4Codes + g) | (lds_u8(vb_lane + o + kKv4Codes + g) << 8);
      if (stored < 64) {
        if (ta + tok + r >= stored) f[r] &= 0xFF00u;
        if (tb + tok + r >= stored) f[r] &= 0x00FFu;
      }
      f[r] = kv4_scales(f[r]);
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint32_t a[2][2][4];  // [token pair][even, odd elements][byte]
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t x = w ? xa[r].y : xa[r].x, y = w ? xb[r].y : xb[r].x;
        e2m1x8_to_f16(select_bits(x, y << 4, 0x0F0F0F0Fu), a[r][0]);
        e2m1x8_to_f16(select_bits(x >> 4, y, 0x0F0F0F0Fu), a[r][1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[r][0][i] = mul_f16x2(a[r][0][i], f[r]);
          a[r][1][i] = mul_f16x2(a[r][1][i], f[r]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        mma_f16(acc[4 * w + i], a[0][0][i], a[0][1][i], a[1][0][i], a[1][1][i], pb[kt][0], pb[kt][1]);
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    kv4_decode_kernel(const __grid_constant__ Kv4DecodeParams p) {
  using C = Cfg;
  constexpr int STAGES = C::kStages, kGroups = C::kGroups;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) &
                                             ~uintptr_t(127));
  const uint32_t smem_base = smem_u32(smem);
  const uint32_t bar_full = smem_base + C::kBarOff;
  const uint32_t bar_empty = bar_full + 8 * STAGES;
  const uint32_t bar_pfull = bar_empty + 8 * STAGES;
  const uint32_t bar_pfree = bar_pfull + 8 * kPieceQ;
  const uint32_t bar_dfull = bar_pfree + 8 * kPieceQ;
  const uint32_t bar_dfree = bar_dfull + 8 * C::kBufs;
  int* desc = reinterpret_cast<int*>(smem + C::kDescOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff);
  volatile int* s_bad = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 8);
  volatile int* s_last = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 16);
  const unsigned long long book_ns = p.timeout_ns * kBookkeepingWaits;
  int32_t* warp_tot = reinterpret_cast<int32_t*>(smem + C::kMiscOff + 128);
  int32_t* cu = reinterpret_cast<int32_t*>(smem + C::kPlanOff);  // units of a KV head ahead of b

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int B = p.num_seqs, G = (int)gridDim.x;
  const uint32_t H = (uint32_t)p.num_kv_heads;

  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar_full + 8 * s, 2);  // K and V
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int s = 0; s < kPieceQ; ++s) {
      mbar_init(bar_pfull + 8 * s, 1);
      mbar_init(bar_pfree + 8 * s, kConsumerWarps + kEpilogueWarps);
    }
    for (int e = 0; e < C::kBufs; ++e) {
      mbar_init(bar_dfull + 8 * e, kConsumerWarps);
      mbar_init(bar_dfree + 8 * e, kEpilogueWarps);
    }
    *abort_flag = 0;
    *s_bad = 0;
    cu[0] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();

  plan_step<kPairCost>(p, cu, s_bad, warp_tot, kThreads, warp == kProducerWarp);

  if (warp >= kProducerWarp) {
    regs_dec<C::kRegsProducer>();
    if (warp != kProducerWarp) {
      named_bar_sync(3, kThreads);
      return;
    }
    // ------------------------------------------------------------ producer
    const PartPlan M = part_plan<kMinPart>(p, cu, s_bad);
    UnitCopies<STAGES, C::kBatch> copies;
    copies.ring = smem_base;
    copies.full = bar_full;
    copies.empty = bar_empty;
    copies.policy = evict_first_policy();
    copies.abort_flag = abort_flag;
    copies.stop = p.withhold_copies != 0;  // failure-path test: no copy is issued
    bool lost = false;                     // the consumers stopped taking pieces
    int j = 0;
    if (blockIdx.x == 0 && lane == 0 && *s_bad) atomicOr(p.err, HPC_DEVCHK_BAD_LENGTH);
    // A piece's descriptor and, with it, its rows of q.
    const bool q_whole = p.q_sh == kHeadDim;  // 8 rows in one piece of memory
    auto publish = [&](const Piece& x) {
      const int qs = j % kPieceQ;
      const uint32_t pf = bar_pfull + 8 * qs;
      const bool rows = !(x.flags & kFlagEnd) && !copies.stop;
      if (lane == 0 && !lost) {
        if (!wait_phase(bar_pfree + 8 * qs, ((j / kPieceQ) & 1u) ^ 1u, abort_flag, p.err,
                        book_ns, false)) {
          lost = true;
        } else {
          int4* d = reinterpret_cast<int4*>(desc + qs * kDescInts);
          d[0] = make_int4(x.b, x.h, x.t0, x.t0 + x.n);
          d[1] = make_int4(x.flags, x.slot, (int)(copies.g % kGroups), 0);
          // release: the descriptor is visible to its waiters
          if (rows) mbar_arrive_expect_tx(pf, (uint32_t)(kGroup * kQRow));
          else mbar_arrive(pf);
        }
      }
      lost = __shfl_sync(0xffffffffu, (int)lost, 0) != 0;
      __syncwarp();  // (a shuffle orders no memory: lane 0 has seen the slot's rows read, others copy)
      if (rows && !lost) {
        const uint32_t dq = smem_base + C::kQOff + qs * C::kQBytes;
        const __nv_bfloat16* q0 =
            p.q + (int64_t)x.b * p.q_sb + (int64_t)(x.h * kGroup) * p.q_sh;
        if (q_whole) {
          if (lane == 0) kv4_copy(dq, q0, kGroup * kQRow, pf);
        } else if (lane < kGroup) {
          kv4_copy(dq + lane * kQRow, q0 + (int64_t)lane * p.q_sh, kQRow, pf);
        }
      }
      ++j;
    };
    if (blockIdx.x < M.P) {
      walk_part<kPairCost>(
          M, cu, B, H, (int)blockIdx.x, [&](const Piece& x) { copies.ahead(p, x); },
          [&](const Piece& x) {
            publish(x);
            copies.copy(p, x);
          });
    }
    publish(Piece{0, 0, 0, 0, kFlagEnd, -1});
    named_bar_sync(3, kThreads);
    if (*abort_flag) {
      for (int i = j > kPieceQ ? j - kPieceQ : 0; lane == 0 && !lost && i < j; ++i)
        wait_phase(bar_pfull + 8 * (i % kPieceQ), (i / kPieceQ) & 1u, abort_flag, p.err, 1000000000ull,
                   false);
      copies.drain(p);
    }
    return;
  }

  uint4* dep0 = reinterpret_cast<uint4*>(smem + C::kDepOff);  // [warp][vector][lane]
  if (warp >= kEpilogueWarp0) {
    regs_dec<C::kRegsEpilogue>();
    // ------------------------------------------------------------ epilogue
    // For every piece: join the states of the warps that shared its units, then write the
    // result, or a partial state of a split pair; the piece is counted, and the last of a
    // pair's merges them. Each warp does two of the states' eight slices.
    const int e = warp - kEpilogueWarp0;
    for (int j = 0;; ++j) {
      const int qs = j % kPieceQ, buf = j % C::kBufs;
      bool ok = wait_phase(bar_pfull + 8 * qs, (j / kPieceQ) & 1u, abort_flag, p.err, book_ns, false);
      const int* d = desc + qs * kDescInts;
      const int b = d[0], h = d[1], fl = d[4], slot = d[5], rot = d[6];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_pfree + 8 * qs);
      if (ok && !(fl & kFlagEnd))
        ok = wait_phase(bar_dfull + 8 * buf, (j / C::kBufs) & 1u, abort_flag, p.err, book_ns, false);
      // (the warps leave together: barriers lie between)
      if (any_of(2, kEpilogueWarps * 32, !ok || (fl & kFlagEnd))) break;
      const uint4* dep = dep0 + buf * (C::kDepBytes / 16);
      Kv4Slices st;
      st.clear();
      // the states from the warp that had the piece's first unit on: the order, like each
      // warp's units, is a function of the piece alone
      auto state = [&](int v) -> const uint4* {
        const int from = rot + v < kGroups ? rot + v : rot + v - kGroups;
        return dep + from * (kDepVec * 32) + lane;
      };
      float4 ml[kGroups];
#pragma unroll
      for (int v = 0; v < kGroups; ++v) {
        ml[v] = *reinterpret_cast<const float4*>(state(v) + 4 * 32);
        st.m[0] = fmaxf(st.m[0], ml[v].x);
        st.m[1] = fmaxf(st.m[1], ml[v].y);
      }
#pragma unroll
      for (int v = 0; v < kGroups; ++v) {
        const float w0 = ml[v].z * Kv4Slices::factor(ml[v].x, st.m[0]);
        const float w1 = ml[v].w * Kv4Slices::factor(ml[v].y, st.m[1]);
        st.l[0] += w0;
        st.l[1] += w1;
        const uint4 h4 = state(v)[e * 32];
        const uint32_t hw[4] = {h4.x, h4.y, h4.z, h4.w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float2 o = __half22float2(*reinterpret_cast<const __half2*>(&hw[y]));
          st.acc[y >> 1][2 * (y & 1)] += o.x * w0;
          st.acc[y >> 1][2 * (y & 1) + 1] += o.y * w1;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_dfree + 8 * buf);  // the buffer is free
      if (fl & kFlagWhole) {
        st.write(p, b, h, e, lane);
        continue;
      }
      st.store(p.ws + (int64_t)slot * kKv4PartFloat4 + lane, e);
      // The piece of a split pair counts itself; the last one of a pair joins the states
      // in the owners' order. More than kFan pieces are joined in groups of kFan first,
      // each by its last piece, so that no one reads more than a few dozen states. One
      // acquire-release atomic covers the warps' writes (ordered before it by the barrier)
      // and the other pieces', which the warps read after the second barrier.
      const PartPlan M = part_plan<kMinPart>(p, cu, s_bad);
      const int k = fl >> 8, owner = slot >> 1;
      const uint32_t own = (uint32_t)cu[b] * H + (uint32_t)h * (uint32_t)(cu[b + 1] - cu[b]) + kPairCost;
      const int first = (int)M.owner_of(own);
      // piece i of the pair: the first one can be its part's last, the others are their parts' first
      const int64_t slot0 = 2 * (int64_t)first + (own <= M.start(first) ? 0 : 1);
      auto place = [&](int i) -> float4* {
        return p.ws + (i == 0 ? slot0 : 2 * (int64_t)(first + i)) * kKv4PartFloat4 + lane;
      };
      bool last_level = k <= kFan;
      int at = last_level ? 0 : (owner - first) / kFan * kFan, step = 1;
      int count = k - at < kFan ? k - at : kFan;
      for (;;) {  // (one piece of code for both levels: it runs cold)
        int32_t* cnt = last_level ? p.pair_cnt + (int64_t)b * H + h
                                  : p.slot_cnt + (at == 0 ? slot0 : 2 * (int64_t)(first + at));
        named_bar_sync(2, kEpilogueWarps * 32);
        if (e == 0 && lane == 0) {
          const int arrived = atom_add_acq_rel_gpu(cnt, 1) == count - 1;
          if (arrived) *cnt = 0;  // ready for the next step
          *s_last = arrived;
        }
        named_bar_sync(2, kEpilogueWarps * 32);
        if (!*s_last) break;
        st.clear();
        st.join(count, e, [&](int i) { return place(at + i * step); });
        if (last_level) {
          st.write(p, b, h, e, lane);
          break;
        }
        // (every warp has read the leader's state where it overwrites it: its own slices and,
        // the first warp, all warps' maxima and sums)
        named_bar_sync(2, kEpilogueWarps * 32);
        st.store(place(at), e);
        last_level = true;
        at = 0;
        step = kFan;
        count = (k + kFan - 1) / kFan;
      }
    }
    // sequences without tiles (or a step that cannot be): out = 0, lse = -inf
    for (int b = (int)blockIdx.x * kEpilogueWarps + e; b < B; b += G * kEpilogueWarps) {
      if (!*s_bad && cu[b + 1] != cu[b]) continue;
      for (int x = lane; x < (int)H * kGroup; x += 32) {
        uint4* o = reinterpret_cast<uint4*>(p.out + (int64_t)b * p.o_sb + (int64_t)x * p.o_sh);
#pragma unroll
        for (int i = 0; i < kHeadDim / 8; ++i) o[i] = make_uint4(0u, 0u, 0u, 0u);
        if (p.lse) p.lse[(int64_t)b * p.l_sb + (int64_t)x * p.l_sh] = -INFINITY;
      }
    }
    named_bar_sync(3, kThreads);
    return;
  }

  regs_inc<C::kRegsConsumer>();
  // -------------------------------------------------------------- consumers
  // The warps take the CTA's units in turn, whatever pieces they belong to: a warp's units
  // come to its own slots in its own order, so the parities of its waits are exact. At a
  // piece's end every warp deposits its state; warps wait for each other only at the deposit
  // buffers.
  uint32_t slot = (uint32_t)warp, phase = 0;  // of the warp's next unit
  bool dead = false;
  for (int j = 0;; ++j) {
    const int qs = j % kPieceQ, buf = j % C::kBufs;
    const bool came =
        wait_phase(bar_pfull + 8 * qs, (j / kPieceQ) & 1u, abort_flag, p.err, book_ns, false);
    // no descriptor arrived: the producer is gone (a warp together, whichever lane's time is up)
    if (!__all_sync(0xffffffffu, came)) break;
    const int* d = desc + qs * kDescInts;
    const int b = d[0], t0 = d[2], t1 = d[3], fl = d[4], rot = d[6];
    if (fl & kFlagEnd) break;
    const int n = t1 - t0;
    const int i0 = warp >= rot ? warp - rot : warp - rot + kGroups;  // this warp's first unit
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, acc[8][4];
#pragma unroll
    for (int dm = 0; dm < 8; ++dm) acc[dm][0] = acc[dm][1] = acc[dm][2] = acc[dm][3] = 0.f;
    uint32_t qf[8][2];
    float sl2[2] = {0.f, 0.f};  // factors of the lane's two columns
    int len = 0;
    if (i0 < n) {
      len = __ldg(p.seq_lens + b);
      load_q4(smem_base + C::kQOff + qs * C::kQBytes, lane, qf, sl2);
      // (a factor of 0 would make NaN of masked scores, an infinite one of scores of 0)
#pragma unroll
      for (int x = 0; x < 2; ++x) sl2[x] = fminf(fmaxf(p.score_scale_log2 * sl2[x], FLT_MIN), FLT_MAX);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_pfree + 8 * qs);  // this warp has read the descriptor and q
    for (int i = i0; i < n; i += kGroups) {
      if (!dead) {
        const bool ok = wait_phase(bar_full + 8 * slot, phase, abort_flag, p.err, p.timeout_ns);
        dead = !__all_sync(0xffffffffu, ok);  // warp-uniform decision
      }
      if (!dead) {
        const int stored = len - (t0 + i) * kBlockTokens;
        const uint32_t kb = smem_base + slot * kStage;
        compute_unit4(kb, kb + kKv4Tile, qf, stored, sl2, m, l, acc, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_empty + 8 * slot);
      }
      slot += kGroups;
      if (slot >= STAGES) {
        slot -= STAGES;
        phase ^= 1u;
      }
    }
    // row sums over the 8 lanes sharing a query-head pair
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
      l[1] += __shfl_xor_sync(0xffffffffu, l[1], o);
    }
    // deposit once the epilogue has read the buffer's previous states: o = acc / l in f16
    // (2^-11; |o| is at most the largest |code * scale|, 2688), m and l in fp32
    wait_phase(bar_dfree + 8 * buf, ((j / C::kBufs) & 1u) ^ 1u, abort_flag, p.err, book_ns, false);
    uint4* dep = dep0 + buf * (C::kDepBytes / 16);
    const float v0 = l[0] == 0.f ? 0.f : __fdividef(1.f, l[0]);
    const float v1 = l[1] == 0.f ? 0.f : __fdividef(1.f, l[1]);
    uint4* dw = dep + warp * (kDepVec * 32) + lane;
#pragma unroll
    for (int k = 0; k < 4; ++k)  // slices 2k, 2k + 1
      dw[k * 32] = make_uint4(
          pack_f16(acc[2 * k][0] * v0, acc[2 * k][1] * v1), pack_f16(acc[2 * k][2] * v0, acc[2 * k][3] * v1),
          pack_f16(acc[2 * k + 1][0] * v0, acc[2 * k + 1][1] * v1),
          pack_f16(acc[2 * k + 1][2] * v0, acc[2 * k + 1][3] * v1));
    reinterpret_cast<float4*>(dw)[4 * 32] = make_float4(m[0], m[1], l[0], l[1]);
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_dfull + 8 * buf);  // release to the epilogue
  }
  named_bar_sync(3, kThreads);  // see the producer's exit
}

}  // namespace

cudaError_t launch_kv4_decode(const Kv4DecodeParams& p, int grid, cudaStream_t stream) {
  using C = Cfg;
  if (p.num_seqs > kKv4MaxSeqs || p.q_len != 1) return cudaErrorInvalidValue;
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = once_per_device(configured, [&] {
    return cudaFuncSetAttribute(kv4_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                C::kSmemBytesMax);
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
  return cudaLaunchKernelEx(&cfg, kv4_decode_kernel, p);
}

}  // namespace hpc
