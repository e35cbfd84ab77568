// Gated feed-forward product on CUDA cores and sums of the products' runs, fp32 (see na_glu_fma.cuh).
#include "na_glu_fma.cuh"

namespace na {
namespace glu {
template na_status launch_fma<float>(const GluParams&, Product, const FmaTile&, cudaStream_t);
template na_status launch_sum<float>(const float*, int, long long, long long, void*, void*, cudaStream_t);
}  // namespace glu
}  // namespace na
