// Gated feed-forward product, forward, bf16 (see na_glu_tc.cuh).
#include "na_glu_tc.cuh"

namespace na {
namespace glu {
template na_status launch_tiles<kForward, __nv_bfloat16>(const GluTcParams&, int, cudaStream_t);
template na_status launch_few<kForward, __nv_bfloat16>(const GluTcParams&, int, cudaStream_t);
}  // namespace glu
}  // namespace na
