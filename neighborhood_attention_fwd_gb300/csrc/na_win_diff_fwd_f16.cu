// na_win_diff_fwd_f16.cu -- differential window softmax, forward, f16: kernel instances.
#include "na_win_impl.cuh"

namespace na {
na_status launch_diff_fwd_f16(WinParams& p, cudaStream_t s) { return launch_win_rows<__half, true, false>(p, s); }
}  // namespace na
