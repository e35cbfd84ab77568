// na_win_diff_bwd_f16.cu -- differential window softmax, gradients, f16: kernel instances.
#include "na_win_impl.cuh"

namespace na {
na_status launch_diff_bwd_f16(WinParams& p, cudaStream_t s) { return launch_win_rows<__half, true, true>(p, s); }
}  // namespace na
