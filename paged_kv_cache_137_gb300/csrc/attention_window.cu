// Front end of windowed and block-scaled decode attention: argument checks,
// the split of the visible positions, workspace layout and kernel selection.
#include <algorithm>
#include <atomic>

#include "attention_window.h"
#include "device_common.cuh"

namespace pkv {

// Resident CTAs per SM of the tensor-core kernel (its ring: 64 KiB for rows of
// 256 bytes, 48 KiB for shorter ones; groups above 8 need more registers).
int window_ctas_per_sm(const pkv_kv_desc* d, int group) {
  const int row = d->head_dim * pkv_dtype_bytes(d->kv_dtype);
  return group <= 8 && row < 256 ? 4 : 3;
}

namespace {

constexpr int kMinPart = 1024, kMultiWavePart = 4096;
constexpr int kMaxPart = 1 << 20;   // a multiple of 64

int sm_count() {
  static std::atomic<int> cache[64];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    (void)cudaGetLastError();
    return 152;
  }
  sms = cache[dev].load();
  if (sms > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) {
    (void)cudaGetLastError();
    return 152;
  }
  cache[dev].store(sms);
  return sms;
}

// What a call decides before it launches.
struct WindowPlan {
  int32_t part = 0;     // tokens per split, a multiple of 64
  int64_t seen = 0;     // tokens of the longest span the arguments allow (whole chunks)
  int64_t splits = 1;   // of that span
  bool alike = false;   // most spans are that long: a window over longer contexts
  size_t m_off = 0, l_off = 0, acc_off = 0, bytes = 0;   // workspace (counters first)
};

pkv_status plan_window(const pkv_kv_desc* d, int32_t num_seqs, int32_t num_q_heads, int32_t max_blocks,
                       int32_t window, int32_t sinks, int32_t requested, WindowPlan* out) {
  if (requested < 0) return fail(PKV_ERR_INVALID_ARG, "partition_tokens is negative");
  if (requested % 64 != 0)
    return fail(PKV_ERR_INVALID_ARG, "partition_tokens must be a multiple of 64");
  if (window < 0 || sinks < 0) return fail(PKV_ERR_INVALID_ARG, "window_tokens or sink_tokens is negative");
  if (static_cast<int64_t>(max_blocks) * d->block_size > (int64_t{1} << 30))
    return fail(PKV_ERR_UNSUPPORTED, "context longer than 2^30 tokens");
  WindowPlan p;
  // the most chunks of 16 a query can see: the sinks', and the window's (one
  // more where it starts inside a chunk)
  const int64_t max_ctx = static_cast<int64_t>(max_blocks) * d->block_size;
  int64_t chunks = (max_ctx + 15) / 16;
  if (window > 0)
    chunks = std::min(chunks, (static_cast<int64_t>(sinks) + 15) / 16 + (static_cast<int64_t>(window) + 15) / 16 + 1);
  p.seen = chunks * 16;
  p.alike = window > 0 && max_ctx >= 2 * p.seen;
  if (requested > 0) {
    p.part = requested;
  } else {
    // A merge of splits costs the call about 4 us (partials, a fence, the
    // arrival count, the gather), and a hundred units draw the whole
    // bandwidth, so splits are made for three reasons only:
    //  * fewer (sequence, KV head) pairs than half the SMs: as many splits as
    //    fill the SMs, of at least 1,024 tokens (32 pairs of 4,100 tokens: 19.3
    //    us in four, 29.1 in one; 64 of 1,028: 13.7 us in two, 12.9 in one);
    //  * lengths that vary widely over less than two waves of resident CTAs:
    //    about one wave of units (256 pairs of up to 4,096 tokens: 39 to 41 us
    //    in three, 40 to 42 in one; with longer contexts the longest unit
    //    alone would set the end).  Spans that a window makes alike stay whole
    //    (192 pairs of 2,052 tokens: 35.9 us, 41.3 in two);
    //  * more pairs than two waves: only the longest spans in two (1,024 pairs
    //    of up to 4,096 tokens: 106 us, 111 whole).
    const int64_t sms = sm_count();
    const int64_t slots = sms * window_ctas_per_sm(d, num_q_heads / d->num_kv_heads);
    const int64_t pairs = static_cast<int64_t>(num_seqs) * d->num_kv_heads;
    const int64_t seen = p.seen;
    const bool alike = p.alike;
    int64_t t = seen;
    if (2 * pairs <= sms) {
      const int64_t n = std::max<int64_t>(1, std::min<int64_t>(sms / pairs, seen / kMinPart));
      t = (seen + n - 1) / n;
    } else if (2 * slots <= pairs + 2) {
      t = std::max<int64_t>(kMultiWavePart, (seen + 1) / 2);
    } else if (!alike) {
      // the mean of min(length, seen) over lengths spread evenly up to
      // max_ctx; each pair's last split is half full
      const double mean = static_cast<double>(seen) - 0.5 * static_cast<double>(seen) * seen / std::max<int64_t>(max_ctx, 1);
      const double room = std::max(0.85 * slots - 0.5 * pairs, 0.25 * pairs);
      t = std::max<int64_t>(kMinPart, static_cast<int64_t>(pairs * mean / room) + 1);
    }
    p.part = static_cast<int32_t>(std::min<int64_t>(kMaxPart, (std::max<int64_t>(t, 1) + 63) / 64 * 64));
  }
  const int64_t part_chunks = p.part / 16;
  p.splits = std::max<int64_t>(1, (chunks + part_chunks - 1) / part_chunks);
  if (p.splits > 65535) return fail(PKV_ERR_UNSUPPORTED, "too many splits");
  if (p.splits > 1) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t n = static_cast<size_t>(num_seqs) * num_q_heads * p.splits;
    p.m_off = up(static_cast<size_t>(num_seqs) * d->num_kv_heads * sizeof(int));
    p.l_off = p.m_off + up(n * sizeof(float));
    p.acc_off = p.l_off + up(n * sizeof(float));
    p.bytes = p.acc_off + up(n * d->head_dim * sizeof(float));
  }
  *out = p;
  return PKV_OK;
}

// Whether the tensor-core kernel covers these sizes.
bool window_tc_covers(const pkv_kv_desc* d) {
  if (d->kv_dtype == PKV_F32) return false;
  return static_cast<int64_t>(d->num_blocks) * d->num_kv_heads * d->block_size <= INT32_MAX;
}

pkv_status decode_window_impl(void* out, const void* q, int32_t q_dtype, const void* k_cache,
                              const void* v_cache, const float* block_scales,
                              const int32_t* block_tables, int32_t max_blocks,
                              const int32_t* context_lens, int32_t num_seqs, int32_t num_q_heads,
                              const pkv_kv_desc* desc, int32_t window, int32_t sinks,
                              float softmax_scale, float k_scale, float v_scale,
                              int32_t partition_tokens, void* workspace, size_t workspace_bytes,
                              void* stream) {
  pkv_status st = PKV_OK;
  if (num_seqs < 0 || num_q_heads <= 0 || max_blocks < 0)
    return fail(PKV_ERR_INVALID_ARG, "negative size or no query heads");
  if (num_q_heads % desc->num_kv_heads != 0)
    return fail(PKV_ERR_INVALID_ARG, "num_q_heads must be a multiple of num_kv_heads");
  WindowPlan plan;
  st = plan_window(desc, std::max(num_seqs, 1), num_q_heads, max_blocks, window, sinks, partition_tokens, &plan);
  if (st != PKV_OK) return st;
  if (num_seqs == 0) return PKV_OK;
  if (num_seqs > 65535) return fail(PKV_ERR_UNSUPPORTED, "more than 65535 sequences per call");
  if (max_blocks == 0) return fail(PKV_ERR_INVALID_ARG, "max_blocks is 0");
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens)
    return fail(PKV_ERR_INVALID_ARG, "NULL pointer");
  for (const void* p : {static_cast<const void*>(out), q, k_cache, v_cache})
    if (!aligned(p, 16)) return fail(PKV_ERR_INVALID_ARG, "buffers must be 16-byte aligned");
  if (!aligned(block_tables, 4) || !aligned(context_lens, 4))
    return fail(PKV_ERR_INVALID_ARG, "tables misaligned");
  if (!(softmax_scale == softmax_scale)) return fail(PKV_ERR_INVALID_ARG, "softmax_scale is NaN");
  const int kv = desc->kv_dtype;
  const bool fp8 = kv == PKV_E4M3;
  if (!(fp8 ? (q_dtype == PKV_F16 || q_dtype == PKV_BF16) : q_dtype == kv))
    return fail(PKV_ERR_INVALID_ARG, "unsupported (kv_dtype, q_dtype) pair");
  const int group = num_q_heads / desc->num_kv_heads;
  if (group > 16) return fail(PKV_ERR_UNSUPPORTED, "more than 16 query heads per KV head");
  if (plan.bytes > 0) {
    if (!workspace || workspace_bytes < plan.bytes)
      return fail(PKV_ERR_INVALID_ARG, "workspace missing or smaller than the workspace size call");
    if (!aligned(workspace, 256)) return fail(PKV_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  }
  const int choice = attention_kernel_choice();
  const bool tc = window_tc_covers(desc) && choice != PKV_KERNEL_SIMT;
  if (choice == PKV_KERNEL_TENSOR_CORE && !tc)
    return fail(PKV_ERR_UNSUPPORTED, "the tensor-core kernel does not cover these sizes");
  int* status = device_status_word(&st);
  if (!status) return st;

  WindowArgs a{};
  a.out = out;
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.tables = block_tables;
  a.ctx_lens = context_lens;
  if (plan.bytes > 0) {
    uint8_t* w = static_cast<uint8_t*>(workspace);
    a.counters = reinterpret_cast<int*>(w);
    a.ws_m = reinterpret_cast<float*>(w + plan.m_off);
    a.ws_l = reinterpret_cast<float*>(w + plan.l_off);
    a.ws_acc = reinterpret_cast<float*>(w + plan.acc_off);
  }
  a.max_blocks = max_blocks;
  a.num_seqs = num_seqs;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = desc->num_kv_heads;
  a.group = group;
  a.num_blocks = desc->num_blocks;
  a.block_size = desc->block_size;
  a.partition = plan.part;
  a.part_chunks = plan.part / 16;
  a.max_splits = static_cast<int32_t>(plan.splits);
  const int64_t units = static_cast<int64_t>(num_seqs) * desc->num_kv_heads * plan.splits;
  a.ctas_per_sm = static_cast<int32_t>(std::min<int64_t>((units + sm_count() - 1) / sm_count(), 4));
  // a unit of few chunks gains nothing from more warps, and each adds to the
  // merge (128 tokens: 4.3 us with four, 5.6 with sixteen)
  const int64_t unit_tokens = plan.seen / plan.splits;
  if (unit_tokens <= 256) a.ctas_per_sm = std::max(a.ctas_per_sm, 3);
  else if (unit_tokens <= 512) a.ctas_per_sm = std::max(a.ctas_per_sm, 2);
  // more than one wave of units alike: two CTAs of six warps finish a last
  // unit sooner than one of four left alone (512 units of 1,028 tokens: 49 us,
  // 56 with three CTAs of four)
  else if (plan.alike && units > 3 * static_cast<int64_t>(sm_count())) a.ctas_per_sm = 2;
  // the CUDA-core form has eight warps for up to two CTAs, else four: eight pay
  // from about 28 chunks on (fp32, 295 units of 416 tokens: 24.5 us with four,
  // 27.4 with eight; 64 of 464: 12.0 and 11.0; 128 of 624: 28.4 and 19.6)
  if (!tc && unit_tokens < 448) a.ctas_per_sm = 3;
  const bool tensor_scales = fp8 && !block_scales;
  a.qk_scale = softmax_scale * (tensor_scales ? k_scale : 1.0f) * 1.4426950408889634f;
  a.v_scale = tensor_scales ? v_scale : 1.0f;
  a.head_scales = desc->head_scales;
  a.softmax_scale = softmax_scale;
  a.status = status;
  a.wait_ns = stage_wait_limit_ns();
  a.window = window;
  a.sinks = window > 0 ? sinks : 0;
  a.block_scales = block_scales;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int D = desc->head_dim;
  if (tc) {
    // boxes of 16 rows whatever the block size: the pool as blocks of 16 (rows
    // of 64 bytes in pairs: eight of 128)
    pkv_kv_desc by16 = *desc;
    by16.num_blocks = desc->num_blocks * (desc->block_size / 16);
    by16.block_size = 16;
    if (D * pkv_dtype_bytes(kv) == 64) {
      by16.head_dim = 2 * D;
      by16.block_size = 8;
    }
    CUtensorMap kmap, vmap;
    st = pool_map(&kmap, k_cache, &by16);
    if (st == PKV_OK) st = pool_map(&vmap, v_cache, &by16);
    if (st != PKV_OK) return st;
    switch (kv) {
      case PKV_F16: return launch_window_tc<F16, F16>(a, D, kmap, vmap, s);
      case PKV_BF16: return launch_window_tc<BF16, BF16>(a, D, kmap, vmap, s);
      default:
        return q_dtype == PKV_F16 ? launch_window_tc<E4M3, F16>(a, D, kmap, vmap, s)
                                  : launch_window_tc<E4M3, BF16>(a, D, kmap, vmap, s);
    }
  }
  switch (kv) {
    case PKV_F32: return launch_window_simt<F32, F32>(a, D, s);
    case PKV_F16: return launch_window_simt<F16, F16>(a, D, s);
    case PKV_BF16: return launch_window_simt<BF16, BF16>(a, D, s);
    default:
      return q_dtype == PKV_F16 ? launch_window_simt<E4M3, F16>(a, D, s)
                                : launch_window_simt<E4M3, BF16>(a, D, s);
  }
}

}  // namespace

pkv_status check_block_scales(const pkv_kv_desc* desc, const float* block_scales) {
  if (desc->kv_dtype != PKV_E4M3) return fail(PKV_ERR_INVALID_ARG, "block_scales need an E4M3 cache");
  if (desc->head_scales)
    return fail(PKV_ERR_INVALID_ARG, "block_scales and head_scales exclude each other");
  if (!block_scales || !aligned(block_scales, 8))
    return fail(PKV_ERR_INVALID_ARG, "block_scales is NULL or misaligned");
  return PKV_OK;
}

}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_window_workspace_bytes(int32_t num_seqs, int32_t num_q_heads, int32_t max_blocks,
                                             const pkv_kv_desc* desc, int32_t window_tokens,
                                             int32_t sink_tokens, int32_t partition_tokens) {
  if (check_desc(desc) != PKV_OK || num_seqs <= 0 || num_q_heads <= 0 || max_blocks <= 0) return 0;
  if (num_q_heads % desc->num_kv_heads != 0) return 0;
  WindowPlan p;
  if (plan_window(desc, num_seqs, num_q_heads, max_blocks, window_tokens, sink_tokens, partition_tokens, &p) != PKV_OK)
    return 0;
  return p.bytes;
}

extern "C" pkv_status pkv_attention_decode_window(
    void* out, const void* q, int32_t q_dtype, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int32_t max_blocks, const int32_t* context_lens, int32_t num_seqs,
    int32_t num_q_heads, const pkv_kv_desc* desc, int32_t window_tokens, int32_t sink_tokens,
    float softmax_scale, float k_scale, float v_scale, int32_t partition_tokens, void* workspace,
    size_t workspace_bytes, void* stream) {
  pkv_status st = check_desc(desc);
  if (st != PKV_OK) return st;
  if (window_tokens < 1) return fail(PKV_ERR_INVALID_ARG, "window_tokens must be at least 1");
  return decode_window_impl(out, q, q_dtype, k_cache, v_cache, nullptr, block_tables, max_blocks,
                            context_lens, num_seqs, num_q_heads, desc, window_tokens, sink_tokens,
                            softmax_scale, k_scale, v_scale, partition_tokens, workspace,
                            workspace_bytes, stream);
}

extern "C" pkv_status pkv_attention_decode_block_scaled(
    void* out, const void* q, int32_t q_dtype, const void* k_cache, const void* v_cache,
    const float* block_scales, const int32_t* block_tables, int32_t max_blocks,
    const int32_t* context_lens, int32_t num_seqs, int32_t num_q_heads, const pkv_kv_desc* desc,
    int32_t window_tokens, int32_t sink_tokens, float softmax_scale, int32_t partition_tokens,
    void* workspace, size_t workspace_bytes, void* stream) {
  pkv_status st = check_desc(desc);
  if (st == PKV_OK) st = check_block_scales(desc, block_scales);
  if (st != PKV_OK) return st;
  return decode_window_impl(out, q, q_dtype, k_cache, v_cache, block_scales, block_tables, max_blocks,
                            context_lens, num_seqs, num_q_heads, desc, window_tokens, sink_tokens,
                            softmax_scale, 1.f, 1.f, partition_tokens, workspace, workspace_bytes,
                            stream);
}
