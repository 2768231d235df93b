// Internal declarations of shared-prefix decode attention (prefix_plan_kernel.cu,
// prefix_decode_kernel.cu, prefix_merge_kernel.cu); not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace hpc {

// A query "pair" is one new token of one sequence, i = b * q_len + t: the 8
// query heads of a KV head make it 8 rows of the 128-row MMA tile, 16 pairs a
// tile. A "work row" v is a set of pairs that read the same K / V tiles: up to
// 32 pairs of a group on the group's shared tiles, or the q_len pairs of one
// sequence on its own tiles behind them. Its work units are (KV head, tile),
// head-major; units of all work rows in order, weighted, are cut into parts of
// equal cost, one part per CTA.
constexpr int kPrefixRowPairs = 32;     // pairs of a shared work row (two MMA tiles)
constexpr int kPrefixTilePairs = 16;    // pairs of one MMA tile
constexpr int32_t kPrefixMaxSeqs = 4096;

// Plan words (device int32).
enum PrefixHeader { kPxRows = 0, kPxParts, kPxPad0, kPxPad1, kPrefixHeader };
// A work row's record, 8 words: {first pair, pairs, block table row, first tile},
// {tiles, 1 for a sequence's own tiles (masked at its end), its length, -}. A
// part's first record is kept beside its boundary, one load away.
struct PrefixLayout {
  int32_t cap_seqs = 0, cap_q_len = 0, cap_parts = 0;
  // work rows: shared ones (every group's last may be partly filled), then own ones
  int64_t cap_rows() const {
    return 2LL * cap_seqs + (int64_t)cap_seqs * cap_q_len / kPrefixRowPairs + 1;
  }
  int64_t bound_off() const { return kPrefixHeader; }                       // [parts + 1][2]
  int64_t seq_off() const { return bound_off() + 2LL * (cap_parts + 1); }   // [seqs][2]
  int64_t first_off() const { return (seq_off() + 2LL * cap_seqs + 7) & ~7LL; }  // [parts][8]
  int64_t rec_off() const { return first_off() + 8LL * cap_parts; }              // [rows][8]
  int64_t words() const { return rec_off() + 8 * cap_rows(); }
};

// Partial softmax states, in blocks of the 8 rows of a (pair, KV head):
// o [32 column groups][8 heads] float4 (unnormalised), m and l [8]. A piece
// that starts a (work row, KV head) goes to the block of its pair, shared or
// own; a piece that continues one to its part's blocks.
struct PrefixWorkspace {
  float4* o;
  float* m;      // log2 units
  float* l;
  int64_t own0;  // first block of the own pieces (shared ones start at 0)
  int64_t cont0; // first block of the parts' continuing pieces, 32 per part
};

// What a KV head of a work row costs its CTA, in units of about 10 ns: a fixed part
// (a shared piece's Q and epilogue; its start counts for every part and cancels)
// and each tile. Found by a random search on the geometric mean of 4 to 8 mixed
// batches of each kind (8 to 60 sequences, 512 .. 32768 shared and 1 .. 2048 own
// positions, 1 to 5 groups); before, with a shared piece priced by its latency
// alone (600), mid-sized batches took up to a fifth more (16 x (2048 + 16 .. 256):
// 26.7 against 21.7 us). Own pieces of one new token run as warp pieces and differ
// from those of several.
struct PrefixCosts {
  int32_t shared_fixed, two_tile, one_tile, own_fixed, own_tile;
};
constexpr PrefixCosts kPrefixCosts[2][2] = {  // [e4m3][several new tokens]
    {{330, 100, 71, 18, 68}, {400, 84, 70, 200, 70}},
    {{300, 90, 63, 58, 35}, {600, 83, 56, 390, 80}}};

struct PrefixPlanParams {
  PrefixCosts costs;
  const int32_t* seq_lens;
  const int32_t* cu_groups;     // [G + 1] or null: one group
  const int32_t* prefix_lens;   // [G]
  int32_t num_seqs, num_groups, q_len, num_kv_heads, max_blocks, num_parts;
  int32_t* words;
  int32_t bound_off, seq_off, first_off, rec_off;
  int32_t* err;
};
cudaError_t launch_prefix_plan(const PrefixPlanParams& p, cudaStream_t stream);

struct PrefixParams {
  const int32_t* words;         // plan
  int32_t bound_off, first_off, rec_off;
  const __nv_bfloat16* q;       // [pairs][H_q][128]
  int64_t q_sp, q_sh;           // element strides over pair, head
  const int32_t* block_table;
  int64_t bt_sb;
  int32_t max_blocks;
  int32_t num_kv_heads, num_blocks, q_len;
  int32_t kv_swap;              // KV tensor map dims are (d, head, slot, block)
  PrefixWorkspace ws;
  float score_scale_log2;       // softmax_scale * log2(e) (* k_scale for e4m3)
  int32_t* err;
  unsigned long long timeout_ns;
  int32_t withhold_copies;
};
// tq16 / tqt: maps over q as [pairs][H_q][128], boxes of 64 columns x 8 heads x
// 16 pairs / q_len pairs, 128-byte swizzle.
cudaError_t launch_prefix_decode(const PrefixParams& p, const CUtensorMap& tq16,
                                 const CUtensorMap& tqt, const CUtensorMap& tk,
                                 const CUtensorMap& tv, bool fp8, int num_parts,
                                 cudaStream_t stream);

struct PrefixMergeParams {
  const int32_t* words;
  int32_t bound_off, seq_off, rec_off;
  int32_t num_seqs, num_kv_heads, q_len;
  PrefixWorkspace ws;
  float v_scale;
  __nv_bfloat16* out;           // element strides over sequence, token, head
  int64_t o_sb, o_st, o_sh;
  float* lse;                   // may be null
  int64_t l_sb, l_st, l_sh;
  int32_t* err;
  unsigned long long timeout_ns;
};
cudaError_t launch_prefix_merge(const PrefixMergeParams& p, int num_sms, cudaStream_t stream);

}  // namespace hpc
