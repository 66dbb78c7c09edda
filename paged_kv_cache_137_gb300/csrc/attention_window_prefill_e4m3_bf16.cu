// Instantiation of windowed prefill attention: E4M3 cache, BF16 queries.
#include "attention_window_prefill.cuh"

namespace pkv {
template pkv_status launch_window_prefill<E4M3, BF16>(const WindowPrefillArgs&, int, int32_t,
                                                    const CUtensorMap&, const CUtensorMap&, cudaStream_t);
}  // namespace pkv
