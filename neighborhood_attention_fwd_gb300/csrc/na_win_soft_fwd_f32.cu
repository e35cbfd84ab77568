// na_win_soft_fwd_f32.cu -- window softmax with dropout, forward, f32: kernel instances.
#include "na_win_impl.cuh"

namespace na {
na_status launch_soft_fwd_f32(WinParams& p, cudaStream_t s) { return launch_win_rows<float, false, false>(p, s); }
}  // namespace na
