// na_win_soft_fwd_bf16.cu -- window softmax with dropout, forward, bf16: kernel instances.
#include "na_win_impl.cuh"

namespace na {
na_status launch_soft_fwd_bf16(WinParams& p, cudaStream_t s) { return launch_win_rows<__nv_bfloat16, false, false>(p, s); }
}  // namespace na
