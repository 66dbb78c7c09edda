// Instantiations of windowed decode attention: bf16 cache, bf16 queries.
#include "attention_window_simt.cuh"

namespace pkv {
template pkv_status launch_window_tc<BF16, BF16>(const WindowArgs&, int, const CUtensorMap&,
                                             const CUtensorMap&, cudaStream_t);
template pkv_status launch_window_simt<BF16, BF16>(const WindowArgs&, int, cudaStream_t);
}  // namespace pkv
