// na_win_f32.cu -- the window softmax kernels' f32 instances.
#include "na_win_impl.cuh"

namespace na {
na_status launch_win_f32(WinParams& p, bool diff, bool bwd, cudaStream_t s) { return launch_win_type<float>(p, diff, bwd, s); }
}  // namespace na
