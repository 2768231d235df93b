// C ABI of shared-prefix decode attention. See include/hpc_decode.h.
#include <climits>
#include <cmath>
#include <cstring>
#include <new>
#include <string>

#include "hpc_internal.h"
#include "prefix_decode.h"

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

int64_t workspace_blocks(const PrefixLayout& L, int64_t kv_heads) {
  return 2LL * L.cap_seqs * L.cap_q_len * kv_heads + (int64_t)kPrefixRowPairs * L.cap_parts;
}

// q as [pairs][H_q][128], box 64 columns x 8 heads x `pairs` pairs.
hpc_status make_pair_map(const hpc_tensor* q, int64_t pairs, int64_t stride, int64_t head_stride,
                         int64_t heads, int box_pairs, CUtensorMap* map) {
  auto enc = encode_fn();
  if (!enc) return fail(HPC_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)heads, (cuuint64_t)pairs};
  cuuint64_t strides[2] = {(cuuint64_t)head_stride * 2, (cuuint64_t)stride * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)kGroup, (cuuint32_t)box_pairs};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q->data, dims, strides, box,
                         estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(HPC_ERR_INVALID_ARG,
                "cuTensorMapEncodeTiled rejected q (error " + std::to_string((int)r) + ")");
  return HPC_OK;
}

hpc_status check_ints(const hpc_tensor* t, const char* name, int64_t n) {
  hpc_status st = check_tensor(t, name, 1);
  if (st != HPC_OK) return st;
  if (t->dtype != HPC_I32 || t->shape[0] != n || (n > 1 && t->stride[0] != 1) ||
      !aligned(t->data, 4))
    return fail(HPC_ERR_INVALID_ARG,
                std::string(name) + " must be contiguous device int32 [" + std::to_string(n) + "]");
  return HPC_OK;
}

}  // namespace

extern "C" {

hpc_status hpc_decode_prefix_plan_create(int32_t max_seqs, int32_t max_q_len, int32_t num_sms,
                                         int32_t num_q_heads, hpc_plan_t* plan_out) {
  return guarded([&]() -> hpc_status {
    if (!plan_out) return fail(HPC_ERR_INVALID_ARG, "plan_out is null");
    *plan_out = nullptr;
    if (max_seqs <= 0 || num_sms <= 0 || num_q_heads <= 0 || num_q_heads % kGroup)
      return fail(HPC_ERR_INVALID_ARG,
                  "max_seqs > 0, num_sms > 0 and num_q_heads a multiple of 8 required");
    if (max_q_len < 1 || max_q_len > kMaxQueryTokens)
      return fail(HPC_ERR_UNSUPPORTED, "max_q_len must be between 1 and 8");
    if (max_seqs > kPrefixMaxSeqs || num_sms > 65536 || num_q_heads > 512)
      return fail(HPC_ERR_UNSUPPORTED, "at most " + std::to_string(kPrefixMaxSeqs) +
                                           " sequences, 65536 CTAs and 512 query heads");
    hpc_plan_s* pl = new hpc_plan_s();
    pl->kind = HPC_PLAN_PREFIX;
    pl->num_sms = num_sms;
    pl->max_seqs = max_seqs;
    pl->prefix_q_len = max_q_len;
    pl->ws_heads = num_q_heads;
    PrefixLayout L;
    L.cap_seqs = max_seqs;
    L.cap_q_len = max_q_len;
    L.cap_parts = num_sms;
    pl->ws_floats = workspace_blocks(L, num_q_heads / kGroup) * (8 * kHeadDim + 16);
    cudaError_t e = cudaGetDevice(&pl->device);
    if (e == cudaSuccess) e = cudaMalloc(&pl->d_words, (size_t)L.words() * sizeof(int32_t));
    if (e == cudaSuccess) e = cudaMalloc(&pl->d_err, sizeof(int32_t));
    if (e == cudaSuccess) e = cudaMemset(pl->d_err, 0, sizeof(int32_t));
    if (e == cudaSuccess) e = cudaMalloc(&pl->d_ws, (size_t)pl->ws_floats * sizeof(float));
    if (e != cudaSuccess) {
      hpc_decode_plan_destroy(pl);
      cudaGetLastError();  // a failed allocation must not look like a later launch's error
      return fail(e == cudaErrorMemoryAllocation ? HPC_ERR_OOM : HPC_ERR_CUDA,
                  std::string("prefix plan: ") + cudaGetErrorString(e));
    }
    *plan_out = pl;
    return HPC_OK;
  });
}

hpc_status hpc_decode_prefix_attn(const hpc_tensor* q, const hpc_tensor* k_cache,
                                  const hpc_tensor* v_cache, const hpc_tensor* block_table,
                                  const hpc_tensor* seq_lens, const hpc_tensor* cu_groups,
                                  const hpc_tensor* prefix_lens, hpc_plan_t plan, hpc_tensor* out,
                                  hpc_tensor* lse, float softmax_scale, void* stream) {
  return guarded([&]() -> hpc_status {
    // what every decode call checks of its tensors
    hpc_plan_s any;
    any.num_seqs = q && q->ndim > 0 && q->ndim <= 4 ? (int32_t)q->shape[0] : 0;
    hpc_status st =
        check_decode_args(q, k_cache, v_cache, block_table, seq_lens, &any, out, lse);
    if (st != HPC_OK) return st;
    const bool multi = q->ndim == 4;
    const int64_t B = q->shape[0], T = multi ? q->shape[1] : 1;
    const int64_t Hq = q->shape[q->ndim - 2], H = k_cache->shape[1], NB = k_cache->shape[0];
    if ((st = check_tensor(prefix_lens, "prefix_lens", 1)) != HPC_OK) return st;
    const int64_t G = prefix_lens->shape[0];
    if (G < 1 || G > kPrefixMaxSeqs)
      return fail(HPC_ERR_INVALID_ARG, "prefix_lens must hold 1 to " +
                                           std::to_string(kPrefixMaxSeqs) + " groups");
    if ((st = check_ints(prefix_lens, "prefix_lens", G)) != HPC_OK) return st;
    if (cu_groups && (st = check_ints(cu_groups, "cu_groups", G + 1)) != HPC_OK) return st;
    if (!cu_groups && G != 1)
      return fail(HPC_ERR_INVALID_ARG, "without cu_groups prefix_lens holds one length");
    const int64_t pair_stride = T > 1 ? q->stride[1] : q->stride[0];  // (token to token)
    if (T > 1 && B > 1 && q->stride[0] != T * q->stride[1])
      return fail(HPC_ERR_INVALID_ARG, "q's tokens must be evenly spaced over the batch "
                                       "(stride 0 = q_len * stride 1)");
    if (!(softmax_scale <= 0.f) && !std::isfinite(softmax_scale))
      return fail(HPC_ERR_INVALID_ARG, "softmax_scale must be finite");
    if (!plan || plan->kind != HPC_PLAN_PREFIX)
      return fail(HPC_ERR_INVALID_ARG, "plan must come from hpc_decode_prefix_plan_create");
    if (B > plan->max_seqs || T > plan->prefix_q_len || Hq > plan->ws_heads)
      return fail(HPC_ERR_INVALID_ARG, "the plan was created for fewer sequences, tokens or heads");
    if (B == 0) return HPC_OK;
    if (NB == 0) return fail(HPC_ERR_INVALID_ARG, "k_cache has no blocks");
    if (NB > INT_MAX || block_table->shape[1] > INT_MAX)
      return fail(HPC_ERR_INVALID_ARG, "sizes exceed int32");
    const bool fp8 = k_cache->dtype == HPC_FP8_E4M3;
    const bool has_lse = lse && lse->data;
    // [blocks][heads][64][128], or (the other layout that the checks admit) the
    // slots outside the heads
    const int64_t s_blk = k_cache->stride[0], s_head = k_cache->stride[1],
                  s_slot = k_cache->stride[2];
    const bool swap = !(s_slot >= kHeadDim && s_head >= kBlockTokens * s_slot && s_blk >= H * s_head);
    CUtensorMap tq16, tqt, tk, tv;
    const int64_t hs = q->stride[q->ndim - 2];
    if ((st = make_pair_map(q, B * T, pair_stride, hs, Hq, kPrefixTilePairs, &tq16)) != HPC_OK ||
        (T > 1 && (st = make_pair_map(q, B * T, pair_stride, hs, Hq, (int)T, &tqt)) != HPC_OK) ||
        (st = make_kv_map(k_cache, fp8, swap, &tk)) != HPC_OK ||
        (st = make_kv_map(v_cache, fp8, swap, &tv)) != HPC_OK)
      return st;
    if (T == 1) tqt = tq16;  // own rows of single tokens are read without a map
    PrefixLayout L;
    L.cap_seqs = plan->max_seqs;
    L.cap_q_len = plan->prefix_q_len;
    L.cap_parts = plan->num_sms;
    PrefixWorkspace ws;
    const int64_t blocks = workspace_blocks(L, plan->ws_heads / kGroup);
    ws.o = (float4*)plan->d_ws;
    ws.m = plan->d_ws + blocks * 8 * kHeadDim;
    ws.l = ws.m + blocks * 8;
    ws.own0 = B * T * H;
    ws.cont0 = 2 * B * T * H;
    const cudaStream_t s = (cudaStream_t)stream;

    PrefixPlanParams pp;
    std::memset(&pp, 0, sizeof pp);
    pp.costs = kPrefixCosts[fp8][T > 1];
    pp.seq_lens = (const int32_t*)seq_lens->data;
    pp.cu_groups = cu_groups ? (const int32_t*)cu_groups->data : nullptr;
    pp.prefix_lens = (const int32_t*)prefix_lens->data;
    pp.num_seqs = (int32_t)B;
    pp.num_groups = (int32_t)G;
    pp.q_len = (int32_t)T;
    pp.num_kv_heads = (int32_t)H;
    pp.max_blocks = (int32_t)block_table->shape[1];
    pp.num_parts = plan->num_sms;
    pp.words = plan->d_words;
    pp.bound_off = (int32_t)L.bound_off();
    pp.seq_off = (int32_t)L.seq_off();
    pp.first_off = (int32_t)L.first_off();
    pp.rec_off = (int32_t)L.rec_off();
    pp.err = plan->d_err;
    cudaError_t e = launch_prefix_plan(pp, s);
    if (e != cudaSuccess)
      return fail(HPC_ERR_CUDA, std::string("prefix planner launch: ") + cudaGetErrorString(e));

    PrefixParams p;
    std::memset(&p, 0, sizeof p);
    p.words = plan->d_words;
    p.q = (const __nv_bfloat16*)q->data;
    p.q_sp = pair_stride;
    p.q_sh = hs;
    p.bound_off = pp.bound_off;
    p.first_off = pp.first_off;
    p.rec_off = pp.rec_off;
    p.block_table = (const int32_t*)block_table->data;
    p.bt_sb = block_table->stride[0];
    p.max_blocks = pp.max_blocks;
    p.num_kv_heads = (int32_t)H;
    p.num_blocks = (int32_t)NB;
    p.q_len = (int32_t)T;
    p.kv_swap = swap;
    p.ws = ws;
    const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt((float)kHeadDim);
    p.score_scale_log2 = scale * 1.4426950408889634f * (fp8 ? k_cache->scale : 1.0f);
    p.err = plan->d_err;
    p.timeout_ns = wait_limit_ns();
    p.withhold_copies = withhold_copies();
    e = launch_prefix_decode(p, tq16, tqt, tk, tv, fp8, plan->num_sms, s);
    if (e != cudaSuccess)
      return fail(HPC_ERR_CUDA, std::string("prefix attention launch: ") + cudaGetErrorString(e));

    PrefixMergeParams mp;
    std::memset(&mp, 0, sizeof mp);
    mp.words = plan->d_words;
    mp.bound_off = pp.bound_off;
    mp.seq_off = pp.seq_off;
    mp.rec_off = pp.rec_off;
    mp.num_seqs = (int32_t)B;
    mp.num_kv_heads = (int32_t)H;
    mp.q_len = (int32_t)T;
    mp.ws = ws;
    mp.v_scale = fp8 ? v_cache->scale : 1.0f;
    mp.out = (__nv_bfloat16*)out->data;
    mp.o_sb = out->stride[0];
    mp.o_st = multi ? out->stride[1] : 0;
    mp.o_sh = out->stride[out->ndim - 2];
    mp.lse = has_lse ? (float*)lse->data : nullptr;
    mp.l_sb = has_lse ? lse->stride[0] : 0;
    mp.l_st = has_lse && multi ? lse->stride[1] : 0;
    mp.l_sh = has_lse ? lse->stride[lse->ndim - 1] : 0;
    mp.err = plan->d_err;
    mp.timeout_ns = wait_limit_ns();
    e = launch_prefix_merge(mp, plan->num_sms, s);
    if (e != cudaSuccess)
      return fail(HPC_ERR_CUDA, std::string("prefix merge launch: ") + cudaGetErrorString(e));
    return HPC_OK;
  });
}

}  // extern "C"
