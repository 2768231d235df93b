// C ABI of the calls that maintain the paged cache: block tables and slot
// maps, rotary positions with the KV write. See include/hpc_decode.h for the contract of every call.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
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

// Rows [tokens][heads] of a fixed number of bytes, strides in bytes.
struct Rows {
  const char* p;
  int64_t n, h, sn, sh, row;
  Rows(const hpc_tensor* t, int64_t elt)
      : p((const char*)t->data), n(t->shape[0]), h(t->shape[1]), sn(t->stride[0] * elt),
        sh(t->stride[1] * elt), row(kHeadDim * elt) {}
  const char* end() const { return p + (n - 1) * sn + (h - 1) * sh + row; }
};

int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b != 0 && (a < 0) != (b < 0)); }

// Whether a row of `a` shares bytes with one of `b` (itself: with another one of its
// rows). Exact for equal strides, as views of one buffer have them. With unequal
// token strides byte ranges that meet count as overlapping, with unequal head
// strides the ranges of a token's rows.
bool rows_overlap(Rows a, Rows b, bool itself = false) {
  if (a.n == 0 || b.n == 0 || a.end() <= b.p || b.end() <= a.p) return false;
  if (a.n == 1) a.sn = b.sn;  // a stride that no row is reached by
  if (b.n == 1) b.sn = a.sn;
  if (a.h == 1) a.sh = b.sh;
  if (b.h == 1) b.sh = a.sh;
  if (a.n == 1 && b.n == 1) a.sn = b.sn = 0;
  if (a.h == 1 && b.h == 1) a.sh = b.sh = 0;
  if (a.sn != b.sn) return true;
  const int64_t sn = a.sn, d = b.p - a.p;
  const int64_t ea = (a.h - 1) * a.sh + a.row, eb = (b.h - 1) * b.sh + b.row;  // a token's extent
  if (itself) {
    if ((a.h == 1 || a.sh >= a.row) && (a.n == 1 || sn >= ea)) return false;
  } else if (sn > 0) {
    const int64_t at = d - floor_div(d, sn) * sn;  // b's tokens behind a's, modulo the stride
    if (ea <= at && at + eb <= sn) return false;
  }
  if (a.sh != b.sh) return true;
  const int64_t sh = a.sh;
  // row (n, h) of a and (n + i, h + j) of b are d + i sn + j sh bytes apart
  for (int64_t j = -(a.h - 1); j < b.h; ++j) {
    const int64_t x = d + j * sh;
    int64_t lo = -(a.n - 1);
    if (sn > 0) lo = std::max(lo, floor_div(-b.row - x, sn) + 1);  // the first with x + i sn > -b.row
    if (itself && j == 0 && lo == 0) ++lo;
    for (int64_t i = lo; i < b.n && x + i * sn < a.row; ++i)
      if (x + i * sn > -b.row && !(itself && i == 0 && j == 0)) return true;
  }
  return false;
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

hpc_status hpc_rope_init(hpc_rope* rope, int32_t rot_dim, int32_t interleaved, double base,
                         int32_t scaling, double factor, int32_t original_len, double low,
                         double high, double magnitude) {
  return guarded([&]() -> hpc_status {
    if (!rope) return fail(HPC_ERR_INVALID_ARG, "rope is null");
    if (rot_dim < 2 || rot_dim > kHeadDim || rot_dim % 2)
      return fail(HPC_ERR_INVALID_ARG, "rot_dim must be even, 2 to 128");
    if (!(base > 1.0) || !std::isfinite(base))
      return fail(HPC_ERR_INVALID_ARG, "base must be finite and above 1");
    if (scaling < HPC_ROPE_NONE || scaling > HPC_ROPE_RAMP)
      return fail(HPC_ERR_INVALID_ARG, "unknown scaling");
    if (!(magnitude >= 0.0) || !std::isfinite(magnitude))
      return fail(HPC_ERR_INVALID_ARG, "magnitude must be finite and >= 0 (0: by the scaling)");
    if (scaling != HPC_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
      return fail(HPC_ERR_INVALID_ARG, "factor must be finite and at least 1");
    if (scaling == HPC_ROPE_BASE && rot_dim == 2)
      return fail(HPC_ERR_INVALID_ARG, "scaling the base needs rot_dim > 2");
    const bool bands = scaling == HPC_ROPE_BANDED || scaling == HPC_ROPE_RAMP;
    if (bands && (original_len <= 0 || !(low > 0.0) || !(high > low) || !std::isfinite(high)))
      return fail(HPC_ERR_INVALID_ARG, "need original_len > 0 and 0 < low < high");
    const double two_pi = 2.0 * 3.14159265358979323846;
    const int R = rot_dim;
    if (scaling == HPC_ROPE_BASE) base *= std::pow(factor, R / (R - 2.0));
    if (!std::isfinite(base))
      return fail(HPC_ERR_INVALID_ARG, "the scaled base must be finite");
    // the pair whose wavelength makes `turns` turns over the trained positions
    auto pair_of = [&](double turns) {
      return R * std::log(original_len / (turns * two_pi)) / (2.0 * std::log(base));
    };
    double ramp_lo = 0.0, ramp_hi = 1.0;
    if (scaling == HPC_ROPE_RAMP) {
      ramp_lo = std::max(0.0, std::floor(pair_of(high)));
      ramp_hi = std::min(R - 1.0, std::ceil(pair_of(low)));
    }
    hpc_rope r;
    std::memset(&r, 0, sizeof r);
    r.rot_dim = R;
    r.interleaved = interleaved != 0;
    double mag = magnitude;
    if (mag == 0.0) mag = scaling == HPC_ROPE_RAMP ? 0.1 * std::log(factor) + 1.0 : 1.0;
    r.magnitude = (float)mag;
    if (!(r.magnitude > 0.f) || !std::isfinite(r.magnitude))
      return fail(HPC_ERR_INVALID_ARG, "magnitude must be in fp32's range");
    for (int i = 0; i < R / 2; ++i) {
      double f = std::pow(base, -2.0 * i / R);
      auto clamp01 = [](double x) { return x < 0.0 ? 0.0 : x > 1.0 ? 1.0 : x; };
      if (scaling == HPC_ROPE_LINEAR) {
        f /= factor;
      } else if (scaling == HPC_ROPE_BANDED) {
        const double keep = clamp01((original_len * f / two_pi - low) / (high - low));
        f = f * keep + f / factor * (1.0 - keep);
      } else if (scaling == HPC_ROPE_RAMP) {
        const double ramp = clamp01((i - ramp_lo) / std::max(ramp_hi - ramp_lo, 0.001));
        f = f / factor * ramp + f * (1.0 - ramp);
      }
      r.freq_hi[i] = (float)f;
      r.freq_lo[i] = (float)(f - (double)r.freq_hi[i]);
    }
    *rope = r;
    return HPC_OK;
  });
}

hpc_status hpc_rope_kv_write(const hpc_tensor* q_in, const hpc_tensor* k_in, const hpc_tensor* v_in,
                             const hpc_tensor* positions, const hpc_tensor* slots,
                             const hpc_rope* rope, const hpc_tensor* q_norm_weight,
                             const hpc_tensor* k_norm_weight, float eps, hpc_tensor* q_out,
                             hpc_tensor* q_out_fp8, hpc_tensor* k_cache, hpc_tensor* v_cache,
                             int32_t* device_error, void* stream) {
  return guarded([&]() -> hpc_status {
    hpc_status st;
    const hpc_tensor* rows[] = {q_in, k_in, v_in, q_out};
    const char* names[] = {"q_in", "k_in", "v_in", "q_out"};
    for (int i = 0; i < 4; ++i)
      if (!empty(rows[i], 3) && (st = check_tensor(rows[i], names[i], 3)) != HPC_OK) return st;
    const int64_t N = q_in->shape[0], Hq = q_in->shape[1], Hkv = k_in->shape[1];
    if ((st = check_vec(positions, "positions", N)) != HPC_OK) return st;
    if ((st = check_vec(slots, "slots", N)) != HPC_OK) return st;
    if ((st = check_tensor(k_cache, "k_cache", 4)) != HPC_OK) return st;
    if ((st = check_tensor(v_cache, "v_cache", 4)) != HPC_OK) return st;
    if ((st = check_tensor(q_norm_weight, "q_norm_weight", 1, true)) != HPC_OK) return st;
    if ((st = check_tensor(k_norm_weight, "k_norm_weight", 1, true)) != HPC_OK) return st;
    const bool has_qf = q_out_fp8 && (q_out_fp8->data || empty(q_out_fp8, 3));
    if (!rope) return fail(HPC_ERR_INVALID_ARG, "rope is null");
    if (rope->rot_dim < 2 || rope->rot_dim > kHeadDim || rope->rot_dim % 2 ||
        (rope->interleaved != 0 && rope->interleaved != 1) || !std::isfinite(rope->magnitude))
      return fail(HPC_ERR_INVALID_ARG, "rope must come from hpc_rope_init");
    for (int i = 0; i < rope->rot_dim / 2; ++i)
      if (!(std::fabs(rope->freq_hi[i]) <= 1.f) || !(std::fabs(rope->freq_lo[i]) <= 1.f))
        return fail(HPC_ERR_INVALID_ARG, "rope must come from hpc_rope_init");
    for (const hpc_tensor* t : rows) {
      if (t->dtype != HPC_BF16)
        return fail(HPC_ERR_INVALID_ARG, "q_in, k_in, v_in and q_out must be bf16");
      if (t->shape[2] != kHeadDim) return fail(HPC_ERR_UNSUPPORTED, "head_dim must be 128");
      if (t->shape[0] != N) return fail(HPC_ERR_INVALID_ARG, "q/k/v/out hold different tokens");
      if (t->stride[2] != 1 || t->stride[0] % 8 || t->stride[1] % 8 || !aligned(t->data, 16))
        return fail(HPC_ERR_INVALID_ARG,
                    "q/k/v/out rows must be contiguous and 16-byte aligned");
    }
    if (k_cache->shape[3] != kHeadDim) return fail(HPC_ERR_UNSUPPORTED, "head_dim must be 128");
    if (k_cache->shape[2] != kBlockTokens)
      return fail(HPC_ERR_UNSUPPORTED, "KV blocks must hold 64 tokens");
    if (Hkv <= 0 || Hq <= 0 || Hq % Hkv || v_in->shape[1] != Hkv || q_out->shape[1] != Hq ||
        k_cache->shape[1] != Hkv)
      return fail(HPC_ERR_INVALID_ARG, "inconsistent heads of q/k/v/out/cache");
    if (Hq > 65536 || Hkv > 65536) return fail(HPC_ERR_UNSUPPORTED, "at most 65536 heads");
    // q may be rotated in place, rows on their own rows; anything else would
    // read what another CTA has written
    const bool in_place = q_out->data == q_in->data &&
                          (N <= 1 || q_out->stride[0] == q_in->stride[0]) &&
                          (Hq == 1 || q_out->stride[1] == q_in->stride[1]);
    const Rows out_rows(q_out, 2);
    if (rows_overlap(out_rows, out_rows, true))
      return fail(HPC_ERR_INVALID_ARG, "rows of q_out overlap");
    if (!in_place && rows_overlap(out_rows, Rows(q_in, 2)))
      return fail(HPC_ERR_INVALID_ARG, "q_out overlaps q_in other than in place (its rows and strides)");
    if (rows_overlap(out_rows, Rows(k_in, 2)) || rows_overlap(out_rows, Rows(v_in, 2)))
      return fail(HPC_ERR_INVALID_ARG, "q_out overlaps k_in or v_in");
    if (has_qf && (q_out_fp8->dtype != HPC_FP8_E4M3 || q_out_fp8->ndim != 3 ||
                   q_out_fp8->shape[0] != N || q_out_fp8->shape[1] != Hq ||
                   q_out_fp8->shape[2] != kHeadDim || q_out_fp8->stride[2] != 1 ||
                   q_out_fp8->stride[0] % 8 || q_out_fp8->stride[1] % 8 ||
                   q_out_fp8->stride[0] < 0 || q_out_fp8->stride[1] < 0 ||
                   !aligned(q_out_fp8->data, 8) || !(q_out_fp8->scale > 0.f) ||
                   !std::isfinite(q_out_fp8->scale)))
      return fail(HPC_ERR_INVALID_ARG, "q_out_fp8 must be e4m3 [N][H_q][128] with a positive scale");
    if (has_qf) {
      const Rows fp8_rows(q_out_fp8, 1);
      if (rows_overlap(fp8_rows, fp8_rows, true))
        return fail(HPC_ERR_INVALID_ARG, "rows of q_out_fp8 overlap");
      for (const hpc_tensor* t : rows)
        if (rows_overlap(fp8_rows, Rows(t, 2)))
          return fail(HPC_ERR_INVALID_ARG, "q_out_fp8 overlaps q_in, k_in, v_in or q_out");
    }
    for (const hpc_tensor* w : {q_norm_weight, k_norm_weight})
      if (w && w->data && ((w->dtype != HPC_BF16 && w->dtype != HPC_F32) ||
                           w->shape[0] != kHeadDim || w->stride[0] != 1 || !aligned(w->data, 16)))
        return fail(HPC_ERR_INVALID_ARG,
                    "norm weights must be contiguous bf16/f32 [128], 16-B aligned");
    if (!(eps >= 0.f) || !std::isfinite(eps))
      return fail(HPC_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (k_cache->dtype != v_cache->dtype ||
        (k_cache->dtype != HPC_BF16 && k_cache->dtype != HPC_FP8_E4M3))
      return fail(HPC_ERR_INVALID_ARG, "k_cache/v_cache must both be bf16 or both fp8_e4m3");
    const bool fp8 = k_cache->dtype == HPC_FP8_E4M3;
    for (int i = 0; i < 4; ++i)
      if (k_cache->shape[i] != v_cache->shape[i] || k_cache->stride[i] != v_cache->stride[i])
        return fail(HPC_ERR_INVALID_ARG, "k_cache and v_cache must have the same shape and strides");
    const uintptr_t unit = fp8 ? 8 : 16;  // bytes of one store
    if (k_cache->stride[3] != 1 || k_cache->stride[0] % 8 || k_cache->stride[1] % 8 ||
        k_cache->stride[2] % 8 || !aligned(k_cache->data, unit) || !aligned(v_cache->data, unit))
      return fail(HPC_ERR_INVALID_ARG, "cache rows must be contiguous and aligned to 8 elements");
    if (fp8 && (!(k_cache->scale > 0.f) || !(v_cache->scale > 0.f) ||
                !std::isfinite(k_cache->scale) || !std::isfinite(v_cache->scale)))
      return fail(HPC_ERR_INVALID_ARG, "FP8 caches need positive finite scales");
    if (N == 0) return HPC_OK;
    for (const hpc_tensor* c : {k_cache, v_cache}) {
      int64_t last = kHeadDim - 1;
      for (int i = 0; i < 3; ++i) last += std::max<int64_t>(c->shape[i] - 1, 0) * c->stride[i];
      const char* begin = (const char*)c->data;
      const char* end = begin + (last + 1) * (fp8 ? 1 : 2);
      auto inside = [&](const Rows& r) { return r.p < end && begin < r.end(); };
      if (inside(out_rows) || (has_qf && inside(Rows(q_out_fp8, 1))))
        return fail(HPC_ERR_INVALID_ARG, "q_out or q_out_fp8 overlaps a cache");
    }
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
      return fail(HPC_ERR_CUDA, std::string("device query: ") + cudaGetErrorString(e));
    RopeParams p;
    std::memset(&p, 0, sizeof p);
    p.q_in = (const __nv_bfloat16*)q_in->data; p.qi_sn = q_in->stride[0]; p.qi_sh = q_in->stride[1];
    p.k_in = (const __nv_bfloat16*)k_in->data; p.ki_sn = k_in->stride[0]; p.ki_sh = k_in->stride[1];
    p.v_in = (const __nv_bfloat16*)v_in->data; p.vi_sn = v_in->stride[0]; p.vi_sh = v_in->stride[1];
    p.positions = (const int32_t*)positions->data;
    p.slots = (const int32_t*)slots->data;
    p.num_tokens = N;
    p.num_q_heads = (int32_t)Hq;
    p.num_kv_heads = (int32_t)Hkv;
    p.num_blocks = (int32_t)(k_cache->shape[0] < INT_MAX ? k_cache->shape[0] : INT_MAX);
    if (q_norm_weight && q_norm_weight->data) {
      p.wq = q_norm_weight->data;
      p.wq_dtype = q_norm_weight->dtype;
    }
    if (k_norm_weight && k_norm_weight->data) {
      p.wk = k_norm_weight->data;
      p.wk_dtype = k_norm_weight->dtype;
    }
    p.eps = eps;
    p.rot_dim = rope->rot_dim;
    p.interleaved = rope->interleaved;
    p.magnitude = rope->magnitude;
    std::memcpy(p.freq_hi, rope->freq_hi, sizeof p.freq_hi);
    std::memcpy(p.freq_lo, rope->freq_lo, sizeof p.freq_lo);
    // 2 pi = 6.28318530717958647692528676655900577; the double holds 53 bits,
    // the third float takes what it leaves out as well
    const double two_pi = 6.283185307179586;         // nearest double
    const double rest = 2.4492935982947064e-16;      // 2 pi minus it
    p.two_pi[0] = (float)two_pi;
    p.two_pi[1] = (float)(two_pi - (double)p.two_pi[0]);
    p.two_pi[2] = (float)(two_pi - (double)p.two_pi[0] - (double)p.two_pi[1] + rest);
    p.q_out = (__nv_bfloat16*)q_out->data; p.qo_sn = q_out->stride[0]; p.qo_sh = q_out->stride[1];
    if (has_qf) {
      p.q_fp8 = (uint8_t*)q_out_fp8->data;
      p.qf_sn = q_out_fp8->stride[0];
      p.qf_sh = q_out_fp8->stride[1];
      p.q_fp8_scale = e4m3_scale(q_out_fp8->scale);
    }
    p.k_cache = k_cache->data;
    p.v_cache = v_cache->data;
    p.c_sblk = k_cache->stride[0]; p.c_shead = k_cache->stride[1]; p.c_sslot = k_cache->stride[2];
    p.cache_fp8 = fp8;
    p.k_scale = e4m3_scale(fp8 ? k_cache->scale : 1.f);
    p.v_scale = e4m3_scale(fp8 ? v_cache->scale : 1.f);
    p.err = device_error;
    e = launch_rope(p, sms, (cudaStream_t)stream);
    if (e != cudaSuccess)
      return fail(HPC_ERR_CUDA, std::string("rope launch: ") + cudaGetErrorString(e));
    return HPC_OK;
  });
}

}  // extern "C"
