// C ABI of the operators around the paged decode: rotary positions, the cache's
// write and read, and latent attention's projections and prompt pass. Argument
// checks and launches only; no call synchronises, allocates or keeps state.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "gqa_kernels.h"
#include "gqa_paged_decode.h"
#include "gqa_rope.cuh"

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxHeadDim = 1024;
constexpr int kMaxHeads = 1024;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool stride_ok(int64_t s, int64_t least, int multiple) { return s >= least && s % multiple == 0; }

// Rotation arguments shared by the entry points; inv_freq == NULL: no rotation.
bool rotation_ok(const int32_t* positions, const double* inv_freq, float scale, int layout) {
  if (inv_freq == nullptr) return true;
  return positions != nullptr && aligned(positions, 4) && aligned(inv_freq, 8) && std::isfinite(scale) &&
         (layout == GQA_ROPE_HALF || layout == GQA_ROPE_INTERLEAVED);
}

int launched(cudaError_t e) { return e == cudaSuccess ? GQA_OK : GQA_ERR_LAUNCH; }

// Packed key rows a prompt pass needs room for: every sequence is rounded up to 128 rows.
int64_t prefill_rows(int batch, int64_t max_kv_tokens) {
  return (max_kv_tokens + 127 * static_cast<int64_t>(batch) + 127) / 128 * 128;
}

bool prefill_sizes_ok(int batch, int num_heads, int64_t max_kv_tokens) {
  return batch > 0 && batch <= (1 << 20) && num_heads > 0 && num_heads <= kMaxHeads && max_kv_tokens >= 0 &&
         max_kv_tokens <= INT32_MAX && prefill_rows(batch, max_kv_tokens) <= INT32_MAX / 2;
}

}  // namespace

extern "C" {

int gqa_rope_inv_freq(int rot_dim, double base, int scaling, double factor, double original_positions, double slow_turns,
                      double fast_turns, double* inv_freq, float* scale) {
  if (rot_dim <= 0 || rot_dim % 2 != 0 || rot_dim > kMaxHeadDim || inv_freq == nullptr) return GQA_ERR_INVALID_ARGUMENT;
  if (!(base > 0.0) || !std::isfinite(base)) return GQA_ERR_INVALID_ARGUMENT;
  if (scaling < GQA_ROPE_SCALING_NONE || scaling > GQA_ROPE_SCALING_BY_PARTS) return GQA_ERR_INVALID_ARGUMENT;
  if (scaling != GQA_ROPE_SCALING_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return GQA_ERR_INVALID_ARGUMENT;
  if (scaling == GQA_ROPE_SCALING_BASE && rot_dim <= 2) return GQA_ERR_INVALID_ARGUMENT;
  if (scaling == GQA_ROPE_SCALING_BY_PARTS &&
      (!(original_positions > 0.0) || !std::isfinite(original_positions) || !(slow_turns >= 0.0) ||
       !(fast_turns > slow_turns) || !std::isfinite(fast_turns)))
    return GQA_ERR_INVALID_ARGUMENT;
  if (scaling == GQA_ROPE_SCALING_BASE) base *= std::pow(factor, rot_dim / (rot_dim - 2.0));
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim);
    if (scaling == GQA_ROPE_SCALING_LINEAR) f /= factor;
    if (scaling == GQA_ROPE_SCALING_BY_PARTS) {
      const double turns = original_positions * f / kTwoPi;
      double keep = (turns - slow_turns) / (fast_turns - slow_turns);
      keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
      f = f * keep + f / factor * (1.0 - keep);
    }
    inv_freq[i] = f;
  }
  if (scale != nullptr)
    *scale = scaling == GQA_ROPE_SCALING_BY_PARTS ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return GQA_OK;
}

int gqa_rope(const void* x, const int32_t* positions, const double* inv_freq, float scale, void* out, int num_tokens,
             int num_heads, int head_dim, int rot_offset, int rot_dim, int layout, int inverse, int dtype,
             int64_t x_token_stride, int64_t x_head_stride, int64_t out_token_stride, int64_t out_head_stride,
             struct CUstream_st* stream) {
  if (num_tokens < 0) return GQA_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return GQA_OK;
  if (x == nullptr || out == nullptr || inv_freq == nullptr) return GQA_ERR_INVALID_ARGUMENT;
  if (!rotation_ok(positions, inv_freq, scale, layout)) return GQA_ERR_INVALID_ARGUMENT;
  if (num_heads <= 0 || num_heads > kMaxHeads || head_dim <= 0 || head_dim > kMaxHeadDim) return GQA_ERR_INVALID_ARGUMENT;
  if (rot_dim <= 0 || rot_dim % 2 != 0 || rot_offset < 0 || rot_offset > head_dim - rot_dim) return GQA_ERR_INVALID_ARGUMENT;
  if (dtype != GQA_TYPE_BF16 && dtype != GQA_TYPE_F16 && dtype != GQA_TYPE_F32) return GQA_ERR_INVALID_ARGUMENT;
  const uintptr_t size = dtype == GQA_TYPE_F32 ? 4 : 2;
  if (!aligned(x, size) || !aligned(out, size)) return GQA_ERR_INVALID_ARGUMENT;
  // rows of the output must not overlap: heads apart within a token, or tokens apart within a head
  if (x_token_stride < 0 || x_head_stride < 0 || out_token_stride < 0 || out_head_stride < 0) return GQA_ERR_INVALID_ARGUMENT;
  const bool token_major = (num_heads == 1 || out_head_stride >= head_dim) &&
                           (num_tokens == 1 || out_token_stride >= (num_heads - 1) * out_head_stride + head_dim);
  const bool head_major = (num_tokens == 1 || out_token_stride >= head_dim) &&
                          (num_heads == 1 || out_head_stride >= (num_tokens - 1) * out_token_stride + head_dim);
  if (!token_major && !head_major) return GQA_ERR_INVALID_ARGUMENT;
  // in place the strides are the same: otherwise rows would be written before others have read them
  if (x == out && ((num_tokens > 1 && x_token_stride != out_token_stride) ||
                   (num_heads > 1 && x_head_stride != out_head_stride)))
    return GQA_ERR_INVALID_ARGUMENT;
  int sms = 0;
  const int rc = gqa::current_device_sms(&sms);
  if (rc != GQA_OK) return rc;
  gqa::RopeParams p{};
  p.x = x;
  p.out = out;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.x_token_stride = x_token_stride;
  p.x_head_stride = x_head_stride;
  p.out_token_stride = out_token_stride;
  p.out_head_stride = out_head_stride;
  p.scale = scale;
  p.num_tokens = num_tokens;
  p.num_heads = num_heads;
  p.head_dim = head_dim;
  p.rot_offset = rot_offset;
  p.rot_dim = rot_dim;
  p.layout = layout;
  p.inverse = inverse != 0;
  return launched(gqa::launch_rope(p, dtype, sms, stream));
}

int gqa_rope_kv_append(const void* q, const void* k_new, const void* v_new, const int32_t* positions,
                       const int32_t* slots, const double* inv_freq, float scale, int rot_offset, int rot_dim, int layout,
                       void* q_out, void* k_cache, void* v_cache, int cache_format, int num_tokens, int num_pages,
                       int64_t q_stride, int64_t k_stride, int64_t v_stride, struct CUstream_st* stream) {
  if (num_tokens < 0) return GQA_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return GQA_OK;
  if (k_new == nullptr || v_new == nullptr || slots == nullptr || k_cache == nullptr || v_cache == nullptr || num_pages <= 0)
    return GQA_ERR_INVALID_ARGUMENT;
  if ((q == nullptr) != (q_out == nullptr)) return GQA_ERR_INVALID_ARGUMENT;
  if (!rotation_ok(positions, inv_freq, scale, layout)) return GQA_ERR_INVALID_ARGUMENT;
  if (inv_freq != nullptr &&
      (rot_dim <= 0 || rot_dim % 2 != 0 || rot_offset < 0 || rot_offset > gqa::kHeadDim - rot_dim))
    return GQA_ERR_INVALID_ARGUMENT;
  if (cache_format != GQA_CACHE_BF16 && cache_format != GQA_CACHE_FP8) return GQA_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(q_out, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(slots, 4))
    return GQA_ERR_INVALID_ARGUMENT;
  const int64_t q_row = gqa::kQoHeads * gqa::kHeadDim, kv_row = gqa::kKvHeads * gqa::kHeadDim;
  if ((q != nullptr && !stride_ok(q_stride, q_row, 8)) || !stride_ok(k_stride, kv_row, 8) ||
      !stride_ok(v_stride, kv_row, 8))
    return GQA_ERR_INVALID_ARGUMENT;
  int sms = 0;
  const int rc = gqa::current_device_sms(&sms);
  if (rc != GQA_OK) return rc;
  gqa::AppendParams p{};
  p.q = q;
  p.k = k_new;
  p.v = v_new;
  p.positions = positions;
  p.slots = slots;
  p.inv_freq = inv_freq;
  p.q_out = q_out;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.scale = scale;
  p.num_tokens = num_tokens;
  p.num_pages = num_pages;
  p.rot_offset = inv_freq != nullptr ? rot_offset : 0;
  p.rot_dim = inv_freq != nullptr ? rot_dim : 0;
  p.layout = inv_freq != nullptr ? layout : GQA_ROPE_HALF;
  p.fp8 = cache_format == GQA_CACHE_FP8;
  return launched(gqa::launch_rope_append(p, sms, stream));
}

int gqa_paged_kv_append_fp8(const void* k_new, const void* v_new, const int32_t* slots, void* k_cache, void* v_cache,
                            int num_tokens, int num_pages, struct CUstream_st* stream) {
  const int64_t row = gqa::kKvHeads * gqa::kHeadDim;
  return gqa_rope_kv_append(nullptr, k_new, v_new, nullptr, slots, nullptr, 1.f, 0, 0, GQA_ROPE_HALF, nullptr, k_cache,
                            v_cache, GQA_CACHE_FP8, num_tokens, num_pages, 0, row, row, stream);
}

int gqa_paged_kv_read_fp8(const void* k_cache, const void* v_cache, const int32_t* indices, void* k_out, void* v_out,
                          int num_tokens, int num_pages, struct CUstream_st* stream) {
  if (num_tokens < 0) return GQA_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return GQA_OK;
  if (k_cache == nullptr || v_cache == nullptr || indices == nullptr || k_out == nullptr || v_out == nullptr ||
      num_pages <= 0)
    return GQA_ERR_INVALID_ARGUMENT;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(indices, 4))
    return GQA_ERR_INVALID_ARGUMENT;
  int sms = 0;
  const int rc = gqa::current_device_sms(&sms);
  if (rc != GQA_OK) return rc;
  return launched(gqa::launch_kv_read_fp8(k_cache, v_cache, indices, k_out, v_out, num_tokens, num_pages, sms, stream));
}

int gqa_mla_kv_append(const void* latent, const void* k_rope, const int32_t* positions, const int32_t* slots,
                      const double* inv_freq, float scale, int layout, void* kv_cache, int num_tokens, int num_slots,
                      int64_t latent_stride, int64_t rope_stride, struct CUstream_st* stream) {
  if (num_tokens < 0) return GQA_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return GQA_OK;
  if (latent == nullptr || k_rope == nullptr || slots == nullptr || kv_cache == nullptr || num_slots <= 0)
    return GQA_ERR_INVALID_ARGUMENT;
  if (!rotation_ok(positions, inv_freq, scale, layout)) return GQA_ERR_INVALID_ARGUMENT;
  if (!aligned(latent, 16) || !aligned(k_rope, 4) || !aligned(kv_cache, 16) || !aligned(slots, 4) ||
      !stride_ok(latent_stride, 512, 8) || !stride_ok(rope_stride, 64, 2))
    return GQA_ERR_INVALID_ARGUMENT;
  int sms = 0;
  const int rc = gqa::current_device_sms(&sms);
  if (rc != GQA_OK) return rc;
  gqa::MlaAppendParams p{};
  p.latent = latent;
  p.k_rope = k_rope;
  p.positions = positions;
  p.slots = slots;
  p.inv_freq = inv_freq;
  p.kv_cache = kv_cache;
  p.latent_stride = latent_stride;
  p.rope_stride = rope_stride;
  p.scale = scale;
  p.num_tokens = num_tokens;
  p.num_slots = num_slots;
  p.layout = inv_freq != nullptr ? layout : GQA_ROPE_HALF;
  return launched(gqa::launch_mla_append(p, sms, stream));
}

int gqa_mla_absorb_q(const void* q, const void* w_kv, const int32_t* positions, const double* inv_freq, float scale,
                     int layout, void* q_out, int num_tokens, int num_heads, int64_t q_token_stride, int64_t q_head_stride,
                     struct CUstream_st* stream) {
  if (num_tokens < 0) return GQA_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return GQA_OK;
  if (q == nullptr || w_kv == nullptr || q_out == nullptr || num_heads <= 0 || num_heads > kMaxHeads ||
      num_tokens > (1 << 20))
    return GQA_ERR_INVALID_ARGUMENT;
  if (!rotation_ok(positions, inv_freq, scale, layout)) return GQA_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(w_kv, 16) || !aligned(q_out, 16) || !stride_ok(q_token_stride, 192, 8) ||
      !stride_ok(q_head_stride, 192, 8))
    return GQA_ERR_INVALID_ARGUMENT;
  int sms = 0;
  gqa::MlaProjParams p{};
  const int rc = gqa::current_device_sms(&sms, &p.wait_limit_ns);
  if (rc != GQA_OK) return rc;
  p.x = q;
  p.w = w_kv;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.out = q_out;
  p.x_token_stride = q_token_stride;
  p.x_head_stride = q_head_stride;
  p.scale = scale;
  p.num_tokens = num_tokens;
  p.num_heads = num_heads;
  p.out_width = 576;
  p.layout = inv_freq != nullptr ? layout : GQA_ROPE_HALF;
  if (gqa::device_error_word(&p.err) != cudaSuccess) return GQA_ERR_LAUNCH;
  return launched(gqa::launch_mla_absorb_q(p, stream));
}

int gqa_mla_expand_out(const void* o_latent, const void* w_kv, void* out, int num_tokens, int num_heads,
                       struct CUstream_st* stream) {
  if (num_tokens < 0) return GQA_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return GQA_OK;
  if (o_latent == nullptr || w_kv == nullptr || out == nullptr || num_heads <= 0 || num_heads > kMaxHeads ||
      num_tokens > (1 << 20))
    return GQA_ERR_INVALID_ARGUMENT;
  if (!aligned(o_latent, 16) || !aligned(w_kv, 16) || !aligned(out, 16)) return GQA_ERR_INVALID_ARGUMENT;
  int sms = 0;
  gqa::MlaProjParams p{};
  const int rc = gqa::current_device_sms(&sms, &p.wait_limit_ns);
  if (rc != GQA_OK) return rc;
  p.x = o_latent;
  p.w = w_kv;
  p.out = out;
  p.x_token_stride = static_cast<int64_t>(num_heads) * 512;
  p.x_head_stride = 512;
  p.num_tokens = num_tokens;
  p.num_heads = num_heads;
  p.out_width = 128;
  if (gqa::device_error_word(&p.err) != cudaSuccess) return GQA_ERR_LAUNCH;
  return launched(gqa::launch_mla_expand_out(p, stream));
}

size_t gqa_mla_prefill_ws_size(int batch, int num_heads, int64_t max_kv_tokens) {
  if (!prefill_sizes_ok(batch, num_heads, max_kv_tokens)) return 0;
  gqa::MlaPrefillParams p{};
  p.batch = batch;
  p.num_heads = num_heads;
  p.cap = static_cast<int>(prefill_rows(batch, max_kv_tokens));
  return gqa::mla_prefill_workspace(&p, nullptr);
}

int gqa_mla_prefill(const void* q, const void* w_kv, const void* kv_cache, const int32_t* block_table,
                    const int32_t* cache_seqlens, const int32_t* cu_seqlens_q, float softmax_scale, int causal, void* out,
                    float* lse, int batch, int total_q, int num_heads, int page_size, int num_blocks, int page_table_width,
                    int64_t max_kv_tokens, int64_t q_token_stride, int64_t q_head_stride, void* workspace,
                    size_t workspace_bytes, struct CUstream_st* stream) {
  return gqa_mla_prefill_fill(q, w_kv, kv_cache, block_table, cache_seqlens, cu_seqlens_q, softmax_scale, causal, 0, out,
                              lse, batch, total_q, num_heads, page_size, num_blocks, page_table_width, max_kv_tokens,
                              q_token_stride, q_head_stride, workspace, workspace_bytes, stream);
}

int gqa_mla_prefill_fill(const void* q, const void* w_kv, const void* kv_cache, const int32_t* block_table,
                         const int32_t* cache_seqlens, const int32_t* cu_seqlens_q, float softmax_scale, int causal,
                         int fill, void* out, float* lse, int batch, int total_q, int num_heads, int page_size,
                         int num_blocks, int page_table_width, int64_t max_kv_tokens, int64_t q_token_stride,
                         int64_t q_head_stride, void* workspace, size_t workspace_bytes, struct CUstream_st* stream) {
  if (batch < 0 || total_q < 0) return GQA_ERR_INVALID_ARGUMENT;
  if (batch == 0 || total_q == 0) return GQA_OK;
  if (!prefill_sizes_ok(batch, num_heads, max_kv_tokens) || total_q > (1 << 26)) return GQA_ERR_INVALID_ARGUMENT;
  if (page_size <= 0 || num_blocks <= 0 || page_table_width <= 0) return GQA_ERR_INVALID_ARGUMENT;
  if (static_cast<int64_t>(num_blocks) * page_size > INT32_MAX || static_cast<int64_t>(page_table_width) * page_size > INT32_MAX)
    return GQA_ERR_INVALID_ARGUMENT;
  if (q == nullptr || w_kv == nullptr || kv_cache == nullptr || block_table == nullptr || cache_seqlens == nullptr ||
      cu_seqlens_q == nullptr || out == nullptr)
    return GQA_ERR_INVALID_ARGUMENT;
  if (fill < 0 || fill > (GQA_FILL_OUT | GQA_FILL_LSE) || ((fill & GQA_FILL_LSE) != 0 && lse == nullptr))
    return GQA_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(softmax_scale * kLog2e)) return GQA_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(w_kv, 16) || !aligned(kv_cache, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(block_table, 4) || !aligned(cache_seqlens, 4) || !aligned(cu_seqlens_q, 4) ||
      !stride_ok(q_token_stride, 192, 8) || !stride_ok(q_head_stride, 192, 8))
    return GQA_ERR_INVALID_ARGUMENT;
  gqa::MlaPrefillParams p{};
  p.q = q;
  p.w = w_kv;
  p.kv = kv_cache;
  p.block_table = block_table;
  p.cache_seqlens = cache_seqlens;
  p.cu_q = cu_seqlens_q;
  p.out = out;
  p.lse = lse;
  p.q_token_stride = q_token_stride;
  p.q_head_stride = q_head_stride;
  p.scale_log2 = softmax_scale * kLog2e;
  p.batch = batch;
  p.total_q = total_q;
  p.num_heads = num_heads;
  p.page_size = page_size;
  p.num_blocks = num_blocks;
  p.width = page_table_width;
  p.causal = causal != 0;
  p.fill = fill;
  p.cap = static_cast<int>(prefill_rows(batch, max_kv_tokens));
  if (workspace == nullptr || !aligned(workspace, 256) ||
      workspace_bytes < gqa::mla_prefill_workspace(&p, static_cast<char*>(workspace)))
    return GQA_ERR_WORKSPACE;
  int sms = 0;
  const int rc = gqa::current_device_sms(&sms);
  if (rc != GQA_OK) return rc;
  if (gqa::device_error_word(&p.err) != cudaSuccess) return GQA_ERR_LAUNCH;
  return launched(gqa::launch_mla_prefill(p, sms, stream));
}

}  // extern "C"
