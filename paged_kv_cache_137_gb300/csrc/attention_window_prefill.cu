// Front end of windowed and block-scaled prefill attention.
#include "attention_window.h"
#include "device_common.cuh"

namespace pkv {
namespace {

pkv_status prefill_window_impl(void* out, const void* q, int32_t q_dtype, const void* k_cache,
                               const void* v_cache, const float* block_scales,
                               const int32_t* block_tables, int32_t max_blocks,
                               const int32_t* context_lens, const int32_t* query_start,
                               int32_t num_seqs, int32_t total_q, int32_t max_query_len,
                               int32_t num_q_heads, const pkv_kv_desc* desc, int32_t window,
                               int32_t sinks, float softmax_scale, float k_scale, float v_scale,
                               void* stream) {
  if (num_seqs < 0 || total_q < 0 || max_query_len < 0 || num_q_heads <= 0 || max_blocks < 0)
    return fail(PKV_ERR_INVALID_ARG, "negative size or no query heads");
  if (window < 0 || sinks < 0) return fail(PKV_ERR_INVALID_ARG, "window_tokens or sink_tokens is negative");
  if (num_q_heads % desc->num_kv_heads != 0)
    return fail(PKV_ERR_INVALID_ARG, "num_q_heads must be a multiple of num_kv_heads");
  if (num_seqs == 0 || total_q == 0 || max_query_len == 0) return PKV_OK;
  if (num_seqs > 65535) return fail(PKV_ERR_UNSUPPORTED, "more than 65535 sequences per call");
  if (max_blocks == 0) return fail(PKV_ERR_INVALID_ARG, "max_blocks is 0");
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start)
    return fail(PKV_ERR_INVALID_ARG, "NULL pointer");
  for (const void* p : {static_cast<const void*>(out), q, k_cache, v_cache})
    if (!aligned(p, 16)) return fail(PKV_ERR_INVALID_ARG, "buffers must be 16-byte aligned");
  if (!aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(query_start, 4))
    return fail(PKV_ERR_INVALID_ARG, "tables misaligned");
  if (static_cast<int64_t>(max_blocks) * desc->block_size > (int64_t{1} << 30))
    return fail(PKV_ERR_UNSUPPORTED, "context longer than 2^30 tokens");
  if (static_cast<int64_t>(desc->num_blocks) * desc->num_kv_heads * desc->block_size > INT32_MAX)
    return fail(PKV_ERR_UNSUPPORTED, "pool larger than 2^31 rows");
  if (!(softmax_scale == softmax_scale)) return fail(PKV_ERR_INVALID_ARG, "softmax_scale is NaN");
  const int kv = desc->kv_dtype;
  const bool fp8 = kv == PKV_E4M3;
  if (!((kv == PKV_BF16 && q_dtype == PKV_BF16) || (kv == PKV_F16 && q_dtype == PKV_F16) ||
        (fp8 && (q_dtype == PKV_F16 || q_dtype == PKV_BF16))))
    return fail(PKV_ERR_UNSUPPORTED, "windowed prefill: 16-bit caches with the same q dtype, or E4M3 with f16/bf16 q");
  pkv_status st = PKV_OK;
  int* status = device_status_word(&st);
  if (!status) return st;

  WindowPrefillArgs a{};
  a.out = out;
  a.q = q;
  a.tables = block_tables;
  a.ctx_lens = context_lens;
  a.query_start = query_start;
  a.max_blocks = max_blocks;
  a.num_seqs = num_seqs;
  a.total_q = total_q;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = desc->num_kv_heads;
  a.group = num_q_heads / desc->num_kv_heads;
  a.num_blocks = desc->num_blocks;
  const bool tensor_scales = fp8 && !block_scales;
  a.qk_scale = softmax_scale * (tensor_scales ? k_scale : 1.0f) * 1.4426950408889634f;
  a.v_scale = tensor_scales ? v_scale : 1.0f;
  a.head_scales = desc->head_scales;
  a.softmax_scale = softmax_scale;
  a.status = status;
  a.window = window;
  a.sinks = window > 0 ? sinks : 0;
  a.block_size = desc->block_size;
  a.block_scales = block_scales;
  // boxes of 16 rows x 128 bytes whatever the block size: the pool as blocks of 16
  pkv_kv_desc by16 = *desc;
  by16.num_blocks = desc->num_blocks * (desc->block_size / 16);
  by16.block_size = 16;
  const int D = desc->head_dim;
  if (fp8 && D != 128)
    return fail(PKV_ERR_UNSUPPORTED, "windowed prefill: E4M3 caches need head_dim 128");
  CUtensorMap kmap, vmap;
  st = pool_map(&kmap, k_cache, &by16, false);
  if (st == PKV_OK) st = pool_map(&vmap, v_cache, &by16, false);
  if (st != PKV_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (kv == PKV_BF16) return launch_window_prefill<BF16, BF16>(a, D, max_query_len, kmap, vmap, s);
  if (kv == PKV_F16) return launch_window_prefill<F16, F16>(a, D, max_query_len, kmap, vmap, s);
  return q_dtype == PKV_F16 ? launch_window_prefill<E4M3, F16>(a, D, max_query_len, kmap, vmap, s)
                            : launch_window_prefill<E4M3, BF16>(a, D, max_query_len, kmap, vmap, s);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_attention_prefill_window(
    void* out, const void* q, int32_t q_dtype, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int32_t max_blocks, const int32_t* context_lens,
    const int32_t* query_start, int32_t num_seqs, int32_t total_q, int32_t max_query_len,
    int32_t num_q_heads, const pkv_kv_desc* desc, int32_t window_tokens, int32_t sink_tokens,
    float softmax_scale, float k_scale, float v_scale, void* stream) {
  const pkv_status st = check_desc(desc);
  if (st != PKV_OK) return st;
  if (window_tokens < 1) return fail(PKV_ERR_INVALID_ARG, "window_tokens must be at least 1");
  return prefill_window_impl(out, q, q_dtype, k_cache, v_cache, nullptr, block_tables, max_blocks,
                             context_lens, query_start, num_seqs, total_q, max_query_len, num_q_heads,
                             desc, window_tokens, sink_tokens, softmax_scale, k_scale, v_scale, stream);
}

extern "C" pkv_status pkv_attention_prefill_block_scaled(
    void* out, const void* q, int32_t q_dtype, const void* k_cache, const void* v_cache,
    const float* block_scales, const int32_t* block_tables, int32_t max_blocks,
    const int32_t* context_lens, const int32_t* query_start, int32_t num_seqs, int32_t total_q,
    int32_t max_query_len, int32_t num_q_heads, const pkv_kv_desc* desc, int32_t window_tokens,
    int32_t sink_tokens, float softmax_scale, void* stream) {
  pkv_status st = check_desc(desc);
  if (st == PKV_OK) st = check_block_scales(desc, block_scales);
  if (st != PKV_OK) return st;
  return prefill_window_impl(out, q, q_dtype, k_cache, v_cache, block_scales, block_tables, max_blocks,
                             context_lens, query_start, num_seqs, total_q, max_query_len, num_q_heads,
                             desc, window_tokens, sink_tokens, softmax_scale, 1.f, 1.f, stream);
}
