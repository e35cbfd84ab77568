// na_win_diff_fwd_f32.cu -- differential window softmax, forward, f32: kernel instances.
#include "na_win_impl.cuh"

namespace na {
na_status launch_diff_fwd_f32(WinParams& p, cudaStream_t s) { return launch_win_rows<float, true, false>(p, s); }
}  // namespace na
