// Gated feed-forward product, forward, fp16 (see na_glu_tc.cuh).
#include "na_glu_tc.cuh"

namespace na {
namespace glu {
template na_status launch_tiles<kForward, __half>(const GluTcParams&, int, cudaStream_t);
template na_status launch_few<kForward, __half>(const GluTcParams&, int, cudaStream_t);
}  // namespace glu
}  // namespace na
