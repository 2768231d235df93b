// C ABI of the calls that maintain the paged cache: block tables and slot
// maps. See include/hpc_decode.h for the contract of every call.
#include <climits>
#include <string>

#include "cache_ops.h"
#include "hpc_internal.h"

using namespace hpc;

namespace {

// Nothing throws across the ABI: a failed host allocation (an error message's
// string) becomes HPC_ERR_OOM.
template <typename F>
hpc_status guarded(F body) noexcept {
  try {
    return body();
  } catch (...) {
    return HPC_ERR_OOM;
  }
}

// A tensor without elements may have a null address.
bool empty(const hpc_tensor* t, int ndim) {
  if (!t || t->ndim != ndim) return false;
  for (int i = 0; i < ndim; ++i)
    if (t->shape[i] == 0) return true;
  return false;
}

hpc_status check_vec(const hpc_tensor* t, const char* name, int64_t n) {
  hpc_status st;
  if (!empty(t, 1) && (st = check_tensor(t, name, 1)) != HPC_OK) return st;
  if (t->dtype != HPC_I32 || (n >= 0 && t->shape[0] != n) || (t->shape[0] > 1 && t->stride[0] != 1))
    return fail(HPC_ERR_INVALID_ARG, std::string(name) + " must be contiguous device int32" +
                                         (n >= 0 ? " [" + std::to_string(n) + "]" : ""));
  if (!aligned(t->data, 4)) return fail(HPC_ERR_INVALID_ARG, std::string(name) + " is misaligned");
  if (t->shape[0] > INT_MAX - 4) return fail(HPC_ERR_INVALID_ARG, std::string(name) + " is too long");
  return HPC_OK;
}

// Byte range of a vector argument, to refuse outputs that lie on inputs.
bool overlap(const hpc_tensor* a, const hpc_tensor* b) {
  const char* x = (const char*)a->data;
  const char* y = (const char*)b->data;
  auto end = [](const hpc_tensor* t) {
    int64_t last = 0;
    for (int i = 0; i < t->ndim; ++i) {
      if (t->shape[i] == 0) return (const char*)t->data;
      last += (t->shape[i] - 1) * t->stride[i];
    }
    return (const char*)t->data + 4 * (last + 1);
  };
  return x < end(b) && y < end(a);
}

// What append and truncate have in common: the lengths, the table and the
// stack of free blocks.
hpc_status check_pool(const hpc_tensor* seq_lens, const hpc_tensor* other, const char* other_name,
                      const hpc_tensor* block_table, const hpc_tensor* free_blocks,
                      const hpc_tensor* free_count, int32_t num_blocks,
                      const hpc_tensor* seq_lens_out, const hpc_tensor* free_count_out) {
  hpc_status st;
  if ((st = check_vec(seq_lens, "seq_lens", -1)) != HPC_OK) return st;
  const int64_t B = seq_lens->shape[0];
  if ((st = check_vec(other, other_name, B)) != HPC_OK) return st;
  if (!empty(block_table, 2) && (st = check_tensor(block_table, "block_table", 2)) != HPC_OK)
    return st;
  if ((st = check_vec(free_blocks, "free_blocks", -1)) != HPC_OK) return st;
  if ((st = check_vec(free_count, "free_count", 1)) != HPC_OK) return st;
  if ((st = check_vec(seq_lens_out, "seq_lens_out", B)) != HPC_OK) return st;
  if ((st = check_vec(free_count_out, "free_count_out", 1)) != HPC_OK) return st;
  if (block_table->dtype != HPC_I32 || block_table->shape[0] != B ||
      (block_table->shape[1] > 1 && block_table->stride[1] != 1) ||
      (B > 1 && block_table->stride[0] < block_table->shape[1]))
    return fail(HPC_ERR_INVALID_ARG,
                "block_table must be int32 [B][max_blocks] with contiguous, separate rows");
  if (block_table->shape[1] > INT_MAX)
    return fail(HPC_ERR_INVALID_ARG, "block_table is too wide");
  if (num_blocks < 0 || num_blocks > INT_MAX / kBlockTokens)
    return fail(HPC_ERR_INVALID_ARG, "num_blocks must be in [0, INT32_MAX / 64]");
  if (B > kBlockTableMaxSeqs)
    return fail(HPC_ERR_UNSUPPORTED, "at most " + std::to_string(kBlockTableMaxSeqs) +
                                         " sequences in one call");
  if (!aligned(block_table->data, 4))
    return fail(HPC_ERR_INVALID_ARG, "block_table is misaligned");
  return HPC_OK;
}

}  // namespace

extern "C" {

hpc_status hpc_block_table_append(const hpc_tensor* seq_lens, const hpc_tensor* new_lens,
                                  const hpc_tensor* free_blocks, const hpc_tensor* free_count,
                                  int32_t num_blocks, hpc_tensor* block_table,
                                  hpc_tensor* seq_lens_out, hpc_tensor* cu_q_lens,
                                  hpc_tensor* positions, hpc_tensor* slots,
                                  hpc_tensor* free_count_out, int32_t* device_error,
                                  void* stream) {
  return guarded([&]() -> hpc_status {
    hpc_status st = check_pool(seq_lens, new_lens, "new_lens", block_table, free_blocks, free_count,
                               num_blocks, seq_lens_out, free_count_out);
    if (st != HPC_OK) return st;
    const int64_t B = seq_lens->shape[0];
    if ((st = check_vec(cu_q_lens, "cu_q_lens", B + 1)) != HPC_OK) return st;
    if ((st = check_vec(positions, "positions", -1)) != HPC_OK) return st;
    if ((st = check_vec(slots, "slots", positions->shape[0])) != HPC_OK) return st;
    const hpc_tensor* outs[] = {seq_lens_out, cu_q_lens, positions, slots, free_count_out,
                                block_table};
    const hpc_tensor* ins[] = {seq_lens, new_lens, free_blocks, free_count};
    for (int i = 0; i < 6; ++i) {
      for (const hpc_tensor* t : ins) {
        const bool in_place = outs[i]->data == t->data &&
                              ((outs[i] == seq_lens_out && t == seq_lens) ||
                               (outs[i] == free_count_out && t == free_count));
        if (!in_place && overlap(outs[i], t))
          return fail(HPC_ERR_INVALID_ARG, "an output overlaps an input");
      }
      for (int j = 0; j < i; ++j)
        if (overlap(outs[i], outs[j]))
          return fail(HPC_ERR_INVALID_ARG, "two outputs overlap");
    }
    AppendParams p;
    p.lens = (const int32_t*)seq_lens->data;
    p.new_lens = (const int32_t*)new_lens->data;
    p.free_blocks = (const int32_t*)free_blocks->data;
    p.free_cap = (int32_t)free_blocks->shape[0];
    p.count = (const int32_t*)free_count->data;
    p.num_blocks = num_blocks;
    p.num_seqs = (int32_t)B;
    p.table = (int32_t*)block_table->data;
    p.bt_sb = block_table->stride[0];
    p.max_blocks = (int32_t)block_table->shape[1];
    p.lens_out = (int32_t*)seq_lens_out->data;
    p.cu = (int32_t*)cu_q_lens->data;
    p.positions = (int32_t*)positions->data;
    p.slots = (int32_t*)slots->data;
    p.cap_tokens = (int32_t)positions->shape[0];
    p.vec4 = aligned(p.positions, 16) && aligned(p.slots, 16);
    p.count_out = (int32_t*)free_count_out->data;
    p.err = device_error;
    const cudaError_t e = launch_append(p, (cudaStream_t)stream);
    if (e != cudaSuccess)
      return fail(HPC_ERR_CUDA, std::string("append launch: ") + cudaGetErrorString(e));
    return HPC_OK;
  });
}

hpc_status hpc_block_table_truncate(const hpc_tensor* seq_lens, const hpc_tensor* to_lens,
                                    const hpc_tensor* block_table, int32_t num_blocks,
                                    hpc_tensor* free_blocks, const hpc_tensor* free_count,
                                    hpc_tensor* seq_lens_out, hpc_tensor* free_count_out,
                                    int32_t* device_error, void* stream) {
  return guarded([&]() -> hpc_status {
    hpc_status st = check_pool(seq_lens, to_lens, "to_lens", block_table, free_blocks, free_count,
                               num_blocks, seq_lens_out, free_count_out);
    if (st != HPC_OK) return st;
    const hpc_tensor* outs[] = {seq_lens_out, free_count_out, free_blocks};
    const hpc_tensor* ins[] = {seq_lens, to_lens, block_table, free_count};
    for (int i = 0; i < 3; ++i) {
      for (const hpc_tensor* t : ins) {
        const bool in_place = outs[i]->data == t->data &&
                              ((outs[i] == seq_lens_out && t == seq_lens) ||
                               (outs[i] == free_count_out && t == free_count));
        if (!in_place && overlap(outs[i], t))
          return fail(HPC_ERR_INVALID_ARG, "an output overlaps an input");
      }
      for (int j = 0; j < i; ++j)
        if (overlap(outs[i], outs[j]))
          return fail(HPC_ERR_INVALID_ARG, "two outputs overlap");
    }
    TruncateParams p;
    p.lens = (const int32_t*)seq_lens->data;
    p.to_lens = (const int32_t*)to_lens->data;
    p.table = (const int32_t*)block_table->data;
    p.bt_sb = block_table->stride[0];
    p.max_blocks = (int32_t)block_table->shape[1];
    p.free_blocks = (int32_t*)free_blocks->data;
    p.free_cap = (int32_t)free_blocks->shape[0];
    p.count = (const int32_t*)free_count->data;
    p.num_blocks = num_blocks;
    p.num_seqs = (int32_t)seq_lens->shape[0];
    p.lens_out = (int32_t*)seq_lens_out->data;
    p.count_out = (int32_t*)free_count_out->data;
    p.err = device_error;
    const cudaError_t e = launch_truncate(p, (cudaStream_t)stream);
    if (e != cudaSuccess)
      return fail(HPC_ERR_CUDA, std::string("truncate launch: ") + cudaGetErrorString(e));
    return HPC_OK;
  });
}

}  // extern "C"
