// na_win_soft_bwd_f16.cu -- window softmax with dropout, gradients, f16: kernel instances.
#include "na_win_impl.cuh"

namespace na {
na_status launch_soft_bwd_f16(WinParams& p, cudaStream_t s) { return launch_win_rows<__half, false, true>(p, s); }
}  // namespace na
