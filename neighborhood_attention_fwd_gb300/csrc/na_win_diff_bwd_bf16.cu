// na_win_diff_bwd_bf16.cu -- differential window softmax, gradients, bf16: kernel instances.
#include "na_win_impl.cuh"

namespace na {
na_status launch_diff_bwd_bf16(WinParams& p, cudaStream_t s) { return launch_win_rows<__nv_bfloat16, true, true>(p, s); }
}  // namespace na
