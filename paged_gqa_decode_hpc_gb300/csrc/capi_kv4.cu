// C ABI of the attention calls over a 4-bit cache (the write is in capi_cache.cu).
// See include/hpc_decode.h for the contract of every call.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <new>
#include <string>

#include "hpc_internal.h"
#include "kv4.cuh"
#include "kv4.h"
#include "prefill.h"

using namespace hpc;

namespace {

template <typename F>
hpc_status guarded(F body) noexcept {
  try {
    return body();
  } catch (...) {  // a failed host allocation must not cross the ABI
    return HPC_ERR_OOM;
  }
}

// A bf16 tensor of rows of 128 elements that kernels read or write 16 bytes at a time.
hpc_status check_rows(const hpc_tensor* t, const char* name, int ndim) {
  if (t->dtype != HPC_BF16) return fail(HPC_ERR_INVALID_ARG, std::string(name) + " must be bf16");
  if (t->shape[ndim - 1] != kHeadDim) return fail(HPC_ERR_UNSUPPORTED, "head_dim must be 128");
  if (t->stride[ndim - 1] != 1)
    return fail(HPC_ERR_INVALID_ARG, std::string(name) + " must have contiguous rows");
  for (int i = 0; i + 1 < ndim; ++i)
    if (t->shape[i] > 1 && t->stride[i] % 8)
      return fail(HPC_ERR_INVALID_ARG, std::string(name) + " must have strides of 8 elements");
  if (!aligned(t->data, 16))
    return fail(HPC_ERR_INVALID_ARG, std::string(name) + " must be 16-byte aligned");
  return HPC_OK;
}

// What a call reads beside q and the caches: lengths and the block table.
hpc_status check_batch(const hpc_tensor* block_table, const hpc_tensor* seq_lens, int64_t B) {
  hpc_status st;
  if ((st = check_tensor(block_table, "block_table", 2)) != HPC_OK) return st;
  if ((st = check_tensor(seq_lens, "seq_lens", 1)) != HPC_OK) return st;
  if (seq_lens->dtype != HPC_I32 || seq_lens->shape[0] != B ||
      (B > 1 && seq_lens->stride[0] != 1) || !aligned(seq_lens->data, 4))
    return fail(HPC_ERR_INVALID_ARG, "seq_lens must be contiguous int32 [B]");
  if (block_table->dtype != HPC_I32 || block_table->shape[0] != B ||
      (block_table->shape[1] > 1 && block_table->stride[1] != 1) || !aligned(block_table->data, 4))
    return fail(HPC_ERR_INVALID_ARG, "block_table must be int32 [B][max_blocks], row-contiguous");
  if (B > INT_MAX || block_table->shape[1] > INT_MAX)
    return fail(HPC_ERR_INVALID_ARG, "sizes exceed int32");
  return HPC_OK;
}

// Whether two tensors' byte ranges meet (element sizes a, b).
bool ranges_meet(const hpc_tensor* x, int64_t a, const hpc_tensor* y, int64_t b) {
  auto end = [](const hpc_tensor* t, int64_t e) {
    int64_t last = 0;
    for (int i = 0; i < t->ndim; ++i) {
      if (t->shape[i] == 0) return (const char*)t->data;
      last += (t->shape[i] - 1) * t->stride[i];
    }
    return (const char*)t->data + (last + 1) * e;
  };
  return (const char*)x->data < end(y, b) && (const char*)y->data < end(x, a);
}

// Whether the first n dimensions of t, over pieces of `inner` elements, lie inside each other
// in some order: then no two pieces meet.
bool nested(const hpc_tensor* t, int n, int64_t inner) {
  int order[4] = {0, 1, 2, 3};
  std::sort(order, order + n, [&](int a, int b) { return t->stride[a] < t->stride[b]; });
  int64_t extent = inner;
  for (int i = 0; i < n; ++i) {
    const int64_t size = t->shape[order[i]], stride = t->stride[order[i]];
    if (size <= 1) continue;
    if (stride < extent) return false;
    extent += (size - 1) * stride;
  }
  return true;
}

// Results of one kind as the checks see them: pieces [sequences][q_len][heads] of a tensor, a row
// of 128 bf16 each or (lse) a float.
struct Pieces {
  const hpc_tensor* t;
  int heads;             // the heads' dimension; [rows][heads] has no tokens of its own
  int64_t elt, inner;    // bytes of an element, elements of a piece
  Pieces(const hpc_tensor* x, bool row)
      : t(x), heads(x->ndim - (row ? 2 : 1)), elt(row ? 2 : 4), inner(row ? kHeadDim : 1) {}
  int64_t tokens() const { return heads == 2 ? t->shape[1] : 1; }
  // [sequences][heads] of one token
  Rows at(int64_t token) const {
    Rows r(t, elt);
    if (heads == 2) r.p += token * t->stride[1] * elt;
    r.h = t->shape[heads];
    r.sh = t->stride[heads] * elt;
    r.row = inner * elt;
    return r;
  }
};

// Whether a piece of a meets one of b: exact where sequences and heads have the same strides
// in both, as in views of one buffer; else byte ranges decide (rows_overlap).
bool pieces_meet(const Pieces& a, const Pieces& b) {
  if (!ranges_meet(a.t, a.elt, b.t, b.elt)) return false;
  for (int64_t i = 0; i < a.tokens(); ++i)
    for (int64_t j = 0; j < b.tokens(); ++j)
      if (rows_overlap(a.at(i), b.at(j))) return true;
  return false;
}

// Whether two of its own pieces meet.
bool pieces_meet(const Pieces& a) {
  if (nested(a.t, a.heads + 1, a.inner)) return false;
  if (rows_overlap(a.at(0), a.at(0), true)) return true;
  for (int64_t i = 1; i < a.tokens(); ++i)
    if (rows_overlap(a.at(0), a.at(i))) return true;
  return false;
}

// out's rows are written while other CTAs read q, in no order: they may not share bytes
// with q's, with each other or with lse.
hpc_status check_overlap(const hpc_tensor* q, const hpc_tensor* out, const hpc_tensor* lse,
                         bool has_lse) {
  const Pieces rq(q, true), ro(out, true);
  if (pieces_meet(ro)) return fail(HPC_ERR_INVALID_ARG, "rows of out overlap");
  if (pieces_meet(ro, rq)) return fail(HPC_ERR_INVALID_ARG, "out overlaps q");
  if (!has_lse) return HPC_OK;
  const Pieces rl(lse, false);
  if (pieces_meet(rl, rq) || pieces_meet(rl, ro))
    return fail(HPC_ERR_INVALID_ARG, "lse overlaps q or out");
  if (pieces_meet(rl)) return fail(HPC_ERR_INVALID_ARG, "elements of lse overlap");
  return HPC_OK;
}

// softmax_scale * log2(e) * K's scale, which has to be a positive float (a value near 0
// or infinity is bounded in the kernels).
hpc_status score_factor(float softmax_scale, float k_scale, float* out) {
  if (!(softmax_scale <= 0.f) && !std::isfinite(softmax_scale))
    return fail(HPC_ERR_INVALID_ARG, "softmax_scale must be finite");
  const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt((float)kHeadDim);
  *out = scale * 1.4426950408889634f * k_scale;
  if (!std::isfinite(*out))
    return fail(HPC_ERR_INVALID_ARG, "softmax_scale times K's scale exceeds fp32");
  return HPC_OK;
}

// q [B][q_len][H_q][128]: a box is 64 columns of the query rows of a KV head.
hpc_status make_kv4_q_map(const hpc_tensor* q, CUtensorMap* map) {
  auto enc = encode_fn();
  if (!enc) return fail(HPC_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const bool multi = q->ndim == 4;
  const int64_t B = q->shape[0], T = multi ? q->shape[1] : 1, Hq = q->shape[q->ndim - 2];
  // (strides of dimensions of one element mean nothing, but have to be multiples of 16 bytes)
  const int64_t sh = q->stride[q->ndim - 2];
  const int64_t st = T > 1 ? q->stride[1] : Hq * kHeadDim, sb = B > 1 ? q->stride[0] : T * Hq * kHeadDim;
  cuuint64_t dims[4] = {(cuuint64_t)kHeadDim, (cuuint64_t)Hq, (cuuint64_t)T, (cuuint64_t)B};
  cuuint64_t strides[3] = {(cuuint64_t)sh * 2, (cuuint64_t)st * 2, (cuuint64_t)sb * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)kGroup, (cuuint32_t)T, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, q->data, dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(HPC_ERR_INVALID_ARG,
                "cuTensorMapEncodeTiled rejected q (error " + std::to_string((int)r) + ")");
  return HPC_OK;
}

int32_t plan_kv_heads(const hpc_plan_s* pl) { return (int32_t)(pl->ws_heads / kGroup); }

}  // namespace

namespace hpc {

hpc_status check_device_memory(const void* data, const char* name) {
  int dev = 0;
  cudaPointerAttributes a;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaPointerGetAttributes(&a, data);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(HPC_ERR_CUDA, std::string("device query: ") + cudaGetErrorString(e));
  }
  if (a.type != cudaMemoryTypeManaged && !(a.type == cudaMemoryTypeDevice && a.device == dev))
    return fail(HPC_ERR_INVALID_ARG, std::string(name) + " is not memory of the current device");
  return HPC_OK;
}

hpc_status check_kv4_caches(const hpc_tensor* k_cache, const hpc_tensor* v_cache) {
  hpc_status st;
  if ((st = check_tensor(k_cache, "k_cache", 4)) != HPC_OK) return st;
  if ((st = check_tensor(v_cache, "v_cache", 4)) != HPC_OK) return st;
  if (k_cache->dtype != HPC_KV4 || v_cache->dtype != HPC_KV4)
    return fail(HPC_ERR_INVALID_ARG, "k_cache/v_cache must be 4-bit rows (HPC_KV4)");
  for (int i = 0; i < 4; ++i)
    if (k_cache->shape[i] != v_cache->shape[i] || k_cache->stride[i] != v_cache->stride[i])
      return fail(HPC_ERR_INVALID_ARG, "k_cache and v_cache must have the same shape and strides");
  if (k_cache->shape[3] != kKv4Row)
    return fail(HPC_ERR_UNSUPPORTED, "a 4-bit row holds a head of 128 in 72 bytes");
  if (k_cache->shape[2] != kBlockTokens)
    return fail(HPC_ERR_UNSUPPORTED, "KV blocks must hold 64 tokens");
  if (k_cache->stride[3] != 1 || k_cache->stride[2] != kKv4Row)
    return fail(HPC_ERR_UNSUPPORTED, "a (block, KV head) tile must be 4608 contiguous bytes");
  if (k_cache->stride[0] % 16 || k_cache->stride[1] % 16 || !aligned(k_cache->data, 16) ||
      !aligned(v_cache->data, 16))
    return fail(HPC_ERR_INVALID_ARG, "tiles must be 16-byte aligned");
  if (!(k_cache->scale > 0.f) || !(v_cache->scale > 0.f) || !std::isfinite(k_cache->scale) ||
      !std::isfinite(v_cache->scale))
    return fail(HPC_ERR_INVALID_ARG, "4-bit caches need positive finite scales");
  return HPC_OK;
}

}  // namespace hpc

extern "C" {

hpc_status hpc_decode_kv4_plan_create(int32_t max_seqs, int32_t max_q_len, int32_t num_sms,
                                      int32_t num_q_heads, hpc_plan_t* plan_out) {
  return guarded([&]() -> hpc_status {
    if (!plan_out) return fail(HPC_ERR_INVALID_ARG, "plan_out is null");
    *plan_out = nullptr;
    if (max_seqs <= 0 || num_sms <= 0 || num_q_heads <= 0 || num_q_heads % kGroup)
      return fail(HPC_ERR_INVALID_ARG,
                  "max_seqs > 0, num_sms > 0 and num_q_heads a multiple of 8 required");
    if (max_q_len < 1 || max_q_len > kMaxQueryTokens)
      return fail(HPC_ERR_UNSUPPORTED, "max_q_len must be between 1 and 8");
    if (max_seqs > kKv4MaxSeqs || num_sms > 65535 || num_q_heads > 512)
      return fail(HPC_ERR_UNSUPPORTED, "at most " + std::to_string(kKv4MaxSeqs) +
                                           " sequences, 65535 CTAs and 512 query heads");
    hpc_plan_s* pl = new hpc_plan_s();
    pl->kind = HPC_PLAN_KV4;
    pl->num_sms = num_sms;
    pl->max_seqs = max_seqs;
    pl->max_q_len = max_q_len;
    pl->ws_heads = num_q_heads;
    pl->ws_floats = kv4_slots(num_sms) * max_q_len * kKv4PartFloat4 * 4;
    const size_t words = (size_t)kv4_words(max_seqs, plan_kv_heads(pl), num_sms);
    cudaError_t e = cudaGetDevice(&pl->device);
    if (e == cudaSuccess) e = cudaMalloc(&pl->d_step, words * sizeof(int32_t));
    if (e == cudaSuccess) e = cudaMemset(pl->d_step, 0, words * sizeof(int32_t));
    if (e == cudaSuccess) e = cudaMalloc(&pl->d_err, sizeof(int32_t));
    if (e == cudaSuccess) e = cudaMemset(pl->d_err, 0, sizeof(int32_t));
    if (e == cudaSuccess) e = cudaMalloc(&pl->d_ws, (size_t)pl->ws_floats * sizeof(float));
    // (cudaMemset is ordered on the legacy stream, the calls on any)
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
    if (e != cudaSuccess) {
      hpc_decode_plan_destroy(pl);
      cudaGetLastError();  // a failed allocation must not look like a later launch's error
      return fail(e == cudaErrorMemoryAllocation ? HPC_ERR_OOM : HPC_ERR_CUDA,
                  std::string("4-bit plan: ") + cudaGetErrorString(e));
    }
    *plan_out = pl;
    return HPC_OK;
  });
}

hpc_status hpc_decode_kv4_attn(const hpc_tensor* q, const hpc_tensor* k_cache,
                               const hpc_tensor* v_cache, const hpc_tensor* block_table,
                               const hpc_tensor* seq_lens, hpc_plan_t plan, hpc_tensor* out,
                               hpc_tensor* lse, float softmax_scale, void* stream) {
  return guarded([&]() -> hpc_status {
    hpc_status st;
    const int nd = q ? q->ndim : 0;
    if (nd != 3 && nd != 4)
      return fail(HPC_ERR_INVALID_ARG, "q must be [B][H_q][128] or [B][q_len][H_q][128]");
    if (q->shape[0] == 0 && out && out->ndim == nd && out->shape[0] == 0)
      return HPC_OK;  // no sequences (null addresses)
    if ((st = check_tensor(q, "q", nd)) != HPC_OK) return st;
    if ((st = check_kv4_caches(k_cache, v_cache)) != HPC_OK) return st;
    if ((st = check_tensor(out, "out", nd)) != HPC_OK) return st;
    if ((st = check_tensor(lse, "lse", nd - 1, true)) != HPC_OK) return st;
    const bool multi = nd == 4, has_lse = lse && lse->data;
    const int64_t B = q->shape[0], T = multi ? q->shape[1] : 1, Hq = q->shape[nd - 2];
    const int64_t NB = k_cache->shape[0], H = k_cache->shape[1];
    if ((st = check_rows(q, "q", nd)) != HPC_OK) return st;
    if ((st = check_rows(out, "out", nd)) != HPC_OK) return st;
    for (int i = 0; i < nd; ++i)
      if (out->shape[i] != q->shape[i])
        return fail(HPC_ERR_INVALID_ARG, "out must have q's shape");
    if (H <= 0 || Hq != kGroup * H)
      return fail(HPC_ERR_UNSUPPORTED, "num_q_heads must be 8 * num_kv_heads");
    if (T < 1 || T > kMaxQueryTokens)
      return fail(HPC_ERR_UNSUPPORTED, "q_len must be between 1 and 8");
    if (has_lse) {
      if (lse->dtype != HPC_F32 || !aligned(lse->data, 4))
        return fail(HPC_ERR_INVALID_ARG, "lse must be f32");
      for (int i = 0; i < nd - 1; ++i)
        if (lse->shape[i] != q->shape[i])
          return fail(HPC_ERR_INVALID_ARG, "lse must be [B][H_q] or [B][q_len][H_q]");
    }
    if ((st = check_batch(block_table, seq_lens, B)) != HPC_OK) return st;
    float factor;
    if ((st = score_factor(softmax_scale, k_cache->scale, &factor)) != HPC_OK) return st;
    if (!plan || plan->kind != HPC_PLAN_KV4)
      return fail(HPC_ERR_INVALID_ARG, "plan must come from hpc_decode_kv4_plan_create");
    if (B > plan->max_seqs || T > plan->max_q_len || Hq > plan->ws_heads)
      return fail(HPC_ERR_INVALID_ARG, "the plan was created for fewer sequences, tokens or heads");
    if (NB == 0) return fail(HPC_ERR_INVALID_ARG, "k_cache has no blocks");
    if (NB > INT_MAX) return fail(HPC_ERR_INVALID_ARG, "sizes exceed int32");
    if ((st = check_overlap(q, out, lse, has_lse)) != HPC_OK) return st;
    if ((st = check_device_memory(out->data, "out")) != HPC_OK) return st;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
      return fail(HPC_ERR_CUDA, std::string("device query: ") + cudaGetErrorString(e));
    if (dev != plan->device)
      return fail(HPC_ERR_INVALID_ARG, "the plan belongs to another device than the current one");

    const int32_t kv_heads = plan_kv_heads(plan);
    Kv4DecodeParams p;
    std::memset(&p, 0, sizeof p);
    p.q = (const __nv_bfloat16*)q->data;
    p.q_sb = q->stride[0];
    p.q_st = multi ? q->stride[1] : 0;
    p.q_sh = q->stride[nd - 2];
    p.out = (__nv_bfloat16*)out->data;
    p.o_sb = out->stride[0];
    p.o_st = multi ? out->stride[1] : 0;
    p.o_sh = out->stride[nd - 2];
    p.lse = has_lse ? (float*)lse->data : nullptr;
    p.l_sb = has_lse ? lse->stride[0] : 0;
    p.l_st = has_lse && multi ? lse->stride[1] : 0;
    p.l_sh = has_lse ? lse->stride[nd - 2] : 0;
    p.k = (const uint8_t*)k_cache->data;
    p.v = (const uint8_t*)v_cache->data;
    p.c_sblk = k_cache->stride[0];
    p.c_shead = k_cache->stride[1];
    p.block_table = (const int32_t*)block_table->data;
    p.bt_sb = block_table->stride[0];
    p.max_blocks = (int32_t)block_table->shape[1];
    p.seq_lens = (const int32_t*)seq_lens->data;
    p.num_seqs = (int32_t)B;
    p.num_kv_heads = (int32_t)H;
    p.num_blocks = (int32_t)NB;
    p.q_len = (int32_t)T;
    p.score_scale_log2 = factor;
    p.v_scale = v_cache->scale;
    p.ws = (float4*)plan->d_ws;
    p.pair_cnt = plan->d_step;
    p.slot_cnt = plan->d_step + kv4_slot_off(plan->max_seqs, kv_heads);
    p.owners = plan->d_step + kv4_owner_off(plan->max_seqs, kv_heads, plan->num_sms);
    p.err = plan->d_err;
    p.timeout_ns = wait_limit_ns();
    p.withhold_copies = withhold_copies();
    p.ws_ml = (float2*)(p.ws + kv4_slots(plan->num_sms) * T * (kGroup * kHeadDim / 4));
    // One token on mma.sync, which has less fixed cost (56 us for 31 x 4096 and 131072 positions
    // of 8 KV heads; the other kernel 77); more on tcgen05, which converts a unit's codes once
    // for all of them (2 tokens 83.6 on mma.sync and 84.3 us, 4: 151.6 and 98.7, 8: 293.5 and
    // 127.8).
    if (T == 1) {
      e = launch_kv4_decode(p, plan->num_sms, (cudaStream_t)stream);
    } else {
      CUtensorMap tq;
      if ((st = make_kv4_q_map(q, &tq)) != HPC_OK) return st;
      e = launch_kv4_tc(p, tq, plan->num_sms, (cudaStream_t)stream);
      if (e == cudaSuccess) e = launch_kv4_merge(p, plan->num_sms, (cudaStream_t)stream);
    }
    if (e != cudaSuccess)
      return fail(HPC_ERR_CUDA, std::string("4-bit decode launch: ") + cudaGetErrorString(e));
    return HPC_OK;
  });
}

hpc_status hpc_extend_kv4_attn(const hpc_tensor* q, const hpc_tensor* k_cache,
                               const hpc_tensor* v_cache, const hpc_tensor* block_table,
                               const hpc_tensor* seq_lens, const hpc_tensor* cu_q_lens,
                               hpc_tensor* out, hpc_tensor* lse, float softmax_scale,
                               int32_t* device_error, void* stream) {
  return guarded([&]() -> hpc_status {
    hpc_status st;
    if (q && out && q->ndim == 3 && out->ndim == 3 && q->shape[0] == 0 && out->shape[0] == 0)
      return HPC_OK;  // no new tokens (null addresses)
    if ((st = check_tensor(q, "q", 3)) != HPC_OK) return st;
    if ((st = check_kv4_caches(k_cache, v_cache)) != HPC_OK) return st;
    if ((st = check_tensor(cu_q_lens, "cu_q_lens", 1)) != HPC_OK) return st;
    if ((st = check_tensor(out, "out", 3)) != HPC_OK) return st;
    if ((st = check_tensor(lse, "lse", 2, true)) != HPC_OK) return st;
    const bool has_lse = lse && lse->data;
    const int64_t N = q->shape[0], Hq = q->shape[1], NB = k_cache->shape[0], H = k_cache->shape[1];
    if ((st = check_rows(q, "q", 3)) != HPC_OK) return st;
    if ((st = check_rows(out, "out", 3)) != HPC_OK) return st;
    for (int i = 0; i < 3; ++i)
      if (out->shape[i] != q->shape[i])
        return fail(HPC_ERR_INVALID_ARG, "out must have q's shape");
    if (H <= 0 || Hq != kGroup * H)
      return fail(HPC_ERR_UNSUPPORTED, "num_q_heads must be 8 * num_kv_heads");
    if (has_lse && (lse->dtype != HPC_F32 || lse->shape[0] != N || lse->shape[1] != Hq ||
                    !aligned(lse->data, 4)))
      return fail(HPC_ERR_INVALID_ARG, "lse must be f32 [total_q][H_q]");
    const int64_t B = cu_q_lens->shape[0] - 1;
    if (cu_q_lens->dtype != HPC_I32 || B < 0 || (B > 0 && cu_q_lens->stride[0] != 1) ||
        !aligned(cu_q_lens->data, 4))
      return fail(HPC_ERR_INVALID_ARG, "cu_q_lens must be contiguous int32 [B+1]");
    if (B == 0) return HPC_OK;
    if ((st = check_batch(block_table, seq_lens, B)) != HPC_OK) return st;
    float factor;
    if ((st = score_factor(softmax_scale, k_cache->scale, &factor)) != HPC_OK) return st;
    if (NB == 0) return fail(HPC_ERR_INVALID_ARG, "k_cache has no blocks");
    if (N > INT_MAX || NB > INT_MAX) return fail(HPC_ERR_INVALID_ARG, "sizes exceed int32");
    if (H > INT_MAX / kGroup) return fail(HPC_ERR_UNSUPPORTED, "too many heads");
    if ((st = check_overlap(q, out, lse, has_lse)) != HPC_OK) return st;
    if ((st = check_device_memory(out->data, "out")) != HPC_OK) return st;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
      return fail(HPC_ERR_CUDA, std::string("device query: ") + cudaGetErrorString(e));
    const int per_cta = extend_tiles_per_cta(N, H, sms);
    const int64_t tokens = (int64_t)kExtendTileTokens * per_cta;
    const int64_t tiles = (N + tokens - 1) / tokens + B;  // sum of ceil(n_b / tokens) at most
    if (tiles > 65535)
      return fail(HPC_ERR_UNSUPPORTED, "too many query tiles in one call (split the batch)");
    CUtensorMap tq, to;
    if ((st = make_q_map(q, &tq, "q")) != HPC_OK) return st;
    if ((st = make_q_map(out, &to, "out")) != HPC_OK) return st;
    ExtendParams p;
    std::memset(&p, 0, sizeof p);
    p.block_table = (const int32_t*)block_table->data;
    p.bt_sb = block_table->stride[0];
    p.max_blocks = (int32_t)block_table->shape[1];
    p.seq_lens = (const int32_t*)seq_lens->data;
    p.cu_q_lens = (const int32_t*)cu_q_lens->data;
    p.num_seqs = (int32_t)B;
    p.num_q_heads = (int32_t)Hq;
    p.num_kv_heads = (int32_t)H;
    p.num_blocks = (int32_t)NB;
    p.out = (__nv_bfloat16*)out->data;
    p.o_st = out->stride[0];
    p.o_sh = out->stride[1];
    p.lse = has_lse ? (float*)lse->data : nullptr;
    p.l_st = has_lse ? lse->stride[0] : 0;
    p.l_sh = has_lse ? lse->stride[1] : 0;
    p.kv_fp8 = 1;
    p.score_scale_log2 = factor;
    p.v_scale = v_cache->scale;
    p.err = device_error;
    p.timeout_ns = wait_limit_ns();
    p.total_q = (int32_t)N;
    p.k4 = (const uint8_t*)k_cache->data;
    p.v4 = (const uint8_t*)v_cache->data;
    p.c_sblk = k_cache->stride[0];
    p.c_shead = k_cache->stride[1];
    p.withhold_copies = withhold_copies();
    e = launch_extend(p, tq, tq, tq, to, (int)tiles, per_cta, (cudaStream_t)stream);
    if (e != cudaSuccess)
      return fail(HPC_ERR_CUDA, std::string("4-bit extend launch: ") + cudaGetErrorString(e));
    return HPC_OK;
  });
}

}  // extern "C"
