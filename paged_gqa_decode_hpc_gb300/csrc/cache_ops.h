// Internal declarations of the operators that maintain the paged cache
// (block_table_kernel.cu, rope_kernel.cu); not part of the public ABI.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

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

}  // namespace hpc
