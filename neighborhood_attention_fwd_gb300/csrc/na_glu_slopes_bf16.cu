// Gated feed-forward product, slopes, bf16 (see na_glu_tc.cuh).
#include "na_glu_tc.cuh"

namespace na {
namespace glu {
template na_status launch_tiles<kSlopes, __nv_bfloat16>(const GluTcParams&, int, cudaStream_t);
template na_status launch_few<kSlopes, __nv_bfloat16>(const GluTcParams&, int, cudaStream_t);
}  // namespace glu
}  // namespace na
