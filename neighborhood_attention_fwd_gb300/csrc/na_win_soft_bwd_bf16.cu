// na_win_soft_bwd_bf16.cu -- window softmax with dropout, gradients, bf16: kernel instances.
#include "na_win_impl.cuh"

namespace na {
na_status launch_soft_bwd_bf16(WinParams& p, cudaStream_t s) { return launch_win_rows<__nv_bfloat16, false, true>(p, s); }
}  // namespace na
