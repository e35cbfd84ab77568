// na_win_f16.cu -- the window softmax kernels' f16 instances.
#include "na_win_impl.cuh"

namespace na {
na_status launch_win_f16(WinParams& p, bool diff, bool bwd, cudaStream_t s) { return launch_win_type<__half>(p, diff, bwd, s); }
}  // namespace na
