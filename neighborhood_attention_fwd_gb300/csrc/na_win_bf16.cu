// na_win_bf16.cu -- the window softmax kernels' bf16 instances.
#include "na_win_impl.cuh"

namespace na {
na_status launch_win_bf16(WinParams& p, bool diff, bool bwd, cudaStream_t s) { return launch_win_type<__nv_bfloat16>(p, diff, bwd, s); }
}  // namespace na
