// na_win_soft_bwd_f32.cu -- window softmax with dropout, gradients, f32: kernel instances.
#include "na_win_impl.cuh"

namespace na {
na_status launch_soft_bwd_f32(WinParams& p, cudaStream_t s) { return launch_win_rows<float, false, true>(p, s); }
}  // namespace na
