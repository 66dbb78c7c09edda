// Instantiations of windowed decode attention: f16 cache, f16 queries.
#include "attention_window_simt.cuh"

namespace pkv {
template pkv_status launch_window_tc<F16, F16>(const WindowArgs&, int, const CUtensorMap&,
                                             const CUtensorMap&, cudaStream_t);
template pkv_status launch_window_simt<F16, F16>(const WindowArgs&, int, cudaStream_t);
}  // namespace pkv
