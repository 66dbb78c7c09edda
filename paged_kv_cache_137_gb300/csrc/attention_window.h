// Internal interface of windowed and block-scaled attention (attention_window.cu,
// attention_window_prefill.cu) and their kernels.
#pragma once

#include "attention.h"

namespace pkv {

// A decode call whose query sees only a window of its context and a few
// first tokens, or whose E4M3 cache has a scale per (block, KV head).
struct WindowArgs : DecodeArgs {
  int32_t window;             // positions [ctx - window, ctx) are seen; 0: all of them
  int32_t sinks;              // and positions [0, sinks)
  int32_t part_chunks;        // 16-token chunks per split
  int32_t ctas_per_sm;        // CTAs of this call that share an SM, at most
  const float* block_scales;  // [num_blocks][N_kv][2] (K, V), or NULL
};

// The tensor-core kernel for one (cache, q) dtype pair.  Defined in
// attention_window_<kv>_<q>.cu through attention_window.cuh.
template <typename KV, typename Q>
pkv_status launch_window_tc(const WindowArgs& a, int head_dim, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, cudaStream_t st);

// The CUDA-core kernel (every dtype pair, head_dim 64 and 128).
template <typename KV, typename Q>
pkv_status launch_window_simt(const WindowArgs& a, int head_dim, cudaStream_t st);

// Prefill with a window, sinks or block scales (attention_window_prefill.cuh).
struct WindowPrefillArgs : PrefillArgs {
  int32_t window, sinks, block_size;
  const float* block_scales;
};
template <typename KV, typename Q>
pkv_status launch_window_prefill(const WindowPrefillArgs& a, int head_dim, int32_t max_query_len,
                                 const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t st);

// The checks a cache with block scales adds.
pkv_status check_block_scales(const pkv_kv_desc* desc, const float* block_scales);

// Resident CTAs per SM of the tensor-core decode kernel.
int window_ctas_per_sm(const pkv_kv_desc* d, int group);

}  // namespace pkv
