// Instantiation of windowed prefill attention: F16 cache, F16 queries.
#include "attention_window_prefill.cuh"

namespace pkv {
template pkv_status launch_window_prefill<F16, F16>(const WindowPrefillArgs&, int, int32_t,
                                                    const CUtensorMap&, const CUtensorMap&, cudaStream_t);
}  // namespace pkv
