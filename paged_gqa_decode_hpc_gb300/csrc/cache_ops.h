// Internal declarations of the operators that maintain the paged cache
// (block_table_kernel.cu, rope_kernel.cu); not part of the public ABI.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "convert.cuh"
#include "hpc_decode.h"

namespace hpc {

// Sequences of one append / truncate call: three int32 per sequence (length,
// two prefix sums) in one CTA's shared memory.
constexpr int32_t kBlockTableMaxSeqs = 16384;

// What one launch of the append kernel writes: everything, the tokens and
// table entries only, or the lengths, their sums and the count only.
enum AppendParts { kAppendAll = 0, kAppendTokens, kAppendLengths };

struct AppendParams {
  const int32_t* lens;          // [B] tokens in the cache
  const int32_t* new_lens;      // [B] tokens to add
  const int32_t* free_blocks;   // [free_cap] stack of free block ids
  int32_t free_cap;
  const int32_t* count;         // [1] ids on the stack
  int32_t num_blocks, num_seqs;
  int32_t* table;               // [B][max_blocks]
  int64_t bt_sb;
  int32_t max_blocks;
  int32_t* lens_out;            // [B], may alias lens
  int32_t* cu;                  // [B + 1]
  int32_t* positions;           // [cap_tokens]
  int32_t* slots;               // [cap_tokens]
  int32_t cap_tokens;
  int32_t vec4;                 // positions and slots are 16-byte aligned
  int32_t* count_out;           // [1], may alias count
  int32_t* err;                 // may be null
  int32_t parts;                // AppendParts, set by launch_append
};
cudaError_t launch_append(const AppendParams& p, cudaStream_t stream);

struct TruncateParams {
  const int32_t* lens;
  const int32_t* to_lens;       // [B] tokens to keep
  const int32_t* table;
  int64_t bt_sb;
  int32_t max_blocks;
  int32_t* free_blocks;         // [free_cap]
  int32_t free_cap;
  const int32_t* count;
  int32_t num_blocks, num_seqs;
  int32_t* lens_out;            // [B], may alias lens
  int32_t* count_out;           // [1], may alias count
  int32_t* err;
};
cudaError_t launch_truncate(const TruncateParams& p, cudaStream_t stream);

// Positions of the rotary kernel are exact in fp32.
constexpr int32_t kRopeMaxPosition = 1 << 24;

struct RopeParams {
  const __nv_bfloat16* q_in;    // [N][H_q][128]; strides in elements over token, head
  int64_t qi_sn, qi_sh;
  const __nv_bfloat16* k_in;
  int64_t ki_sn, ki_sh;
  const __nv_bfloat16* v_in;
  int64_t vi_sn, vi_sh;
  const int32_t* positions;     // [N]
  const int32_t* slots;         // [N], < 0: padding
  int64_t num_tokens;
  int32_t num_q_heads, num_kv_heads, num_blocks;
  const void* wq;               // norm weights, null: no norm
  const void* wk;
  int32_t wq_dtype, wk_dtype;
  float eps;
  int32_t rot_dim, interleaved;
  float magnitude;
  float two_pi[3];              // 2 pi as a sum of floats
  float freq_hi[64], freq_lo[64];
  __nv_bfloat16* q_out;
  int64_t qo_sn, qo_sh;
  uint8_t* q_fp8;               // may be null
  int64_t qf_sn, qf_sh;
  E4m3Scale q_fp8_scale;
  void* k_cache;
  void* v_cache;
  int64_t c_sblk, c_shead, c_sslot;
  int32_t cache_fp8;
  E4m3Scale k_scale, v_scale;
  int32_t* err;                 // may be null
};
cudaError_t launch_rope(const RopeParams& p, int sm_count, cudaStream_t stream);

}  // namespace hpc
