// Gated feed-forward product, gradients of tokens and weights, bf16 (see na_glu_tc.cuh).
#include "na_glu_tc.cuh"

namespace na {
namespace glu {
template na_status launch_tiles<kTokens, __nv_bfloat16>(const GluTcParams&, int, cudaStream_t);
template na_status launch_tiles<kWeights, __nv_bfloat16>(const GluTcParams&, int, cudaStream_t);
template na_status launch_tiles<kBoth, __nv_bfloat16>(const GluTcParams&, int, cudaStream_t);
}  // namespace glu
}  // namespace na
