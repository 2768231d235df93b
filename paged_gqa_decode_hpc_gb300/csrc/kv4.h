// Internal declarations of the attention over a 4-bit cache (kv4_decode_kernel.cu,
// kv4_tc_kernel.cu, kv4_merge_kernel.cu, capi_kv4.cu); not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "hpc_decode.h"

namespace hpc {

// Sequences of one step: their prefix array lies in shared memory.
constexpr int32_t kKv4MaxSeqs = 4096;
// Partial-state slots of a step on `grid` CTAs, each of which owns one part of the units:
// a part's first piece and its last one can be split pairs'.
inline int64_t kv4_slots(int32_t grid) { return 2LL * grid; }
// One token's partial state: 8 accumulator slices and (m, m, l, l) of every lane.
constexpr int kKv4PartFloat4 = 9 * 32;

struct Kv4DecodeParams {
  const __nv_bfloat16* q;       // [B][q_len][H_q][128]
  int64_t q_sb, q_st, q_sh;
  __nv_bfloat16* out;
  int64_t o_sb, o_st, o_sh;
  float* lse;                   // may be null
  int64_t l_sb, l_st, l_sh;
  const uint8_t* k;             // [blocks][H_kv][64][72], strides in bytes
  const uint8_t* v;
  int64_t c_sblk, c_shead;
  const int32_t* block_table;
  int64_t bt_sb;
  int32_t max_blocks;
  const int32_t* seq_lens;
  int32_t num_seqs, num_kv_heads, num_blocks, q_len;
  float score_scale_log2;       // softmax_scale * log2(e) * K's scale, > 0
  float v_scale;
  float4* ws;                   // partial states. One token: [slots][9][32]; several:
                                //   accumulators [slots][q_len][8 heads][32]
  float2* ws_ml;                // (several tokens) maximum, sum [slots][q_len][8]
  int32_t* pair_cnt;            // [B * H_kv] pieces (or groups of them) that have arrived
  int32_t* slot_cnt;            // [slots] pieces of a group that have arrived
  int32_t* owners;              // [4 + 4 owners] (q_len > 1): their number, and of each the pair
                                //   that it begins and others go on with {b, h, pieces, slot}
  int32_t* err;
  unsigned long long timeout_ns;
  int32_t withhold_copies;
};
// int32 words of a plan's counters and records, in the order of the fields above.
inline int64_t kv4_slot_off(int32_t max_seqs, int32_t kv_heads) {
  return (int64_t)max_seqs * kv_heads;
}
inline int64_t kv4_owner_off(int32_t max_seqs, int32_t kv_heads, int32_t grid) {
  return (kv4_slot_off(max_seqs, kv_heads) + kv4_slots(grid) + 3) / 4 * 4;
}
inline int64_t kv4_words(int32_t max_seqs, int32_t kv_heads, int32_t grid) {
  return kv4_owner_off(max_seqs, kv_heads, grid) + 4 + 4LL * grid;
}

// One new token a sequence.
cudaError_t launch_kv4_decode(const Kv4DecodeParams& p, int grid, cudaStream_t stream);
// 2 to 8.
cudaError_t launch_kv4_tc(const Kv4DecodeParams& p, const CUtensorMap& tq, int grid,
                          cudaStream_t stream);
// The split pairs of its step, joined.
cudaError_t launch_kv4_merge(const Kv4DecodeParams& p, int grid, cudaStream_t stream);

}  // namespace hpc
