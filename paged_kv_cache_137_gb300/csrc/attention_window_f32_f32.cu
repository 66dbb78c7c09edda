// Instantiation of windowed decode attention: f32 cache, f32 queries.
#include "attention_window_simt.cuh"

namespace pkv {
template pkv_status launch_window_simt<F32, F32>(const WindowArgs&, int, cudaStream_t);
}  // namespace pkv
