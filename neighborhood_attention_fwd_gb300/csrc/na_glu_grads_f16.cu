// Gated feed-forward product, gradients of tokens and weights, fp16 (see na_glu_tc.cuh).
#include "na_glu_tc.cuh"

namespace na {
namespace glu {
template na_status launch_tiles<kTokens, __half>(const GluTcParams&, int, cudaStream_t);
template na_status launch_tiles<kWeights, __half>(const GluTcParams&, int, cudaStream_t);
template na_status launch_tiles<kBoth, __half>(const GluTcParams&, int, cudaStream_t);
}  // namespace glu
}  // namespace na
