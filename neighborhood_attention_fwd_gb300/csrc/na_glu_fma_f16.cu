// Gated feed-forward product on CUDA cores and sums of the products' runs, fp16 (see na_glu_fma.cuh).
#include "na_glu_fma.cuh"

namespace na {
namespace glu {
template na_status launch_fma<__half>(const GluParams&, Product, const FmaTile&, cudaStream_t);
template na_status launch_sum<__half>(const float*, int, long long, long long, void*, void*, cudaStream_t);
}  // namespace glu
}  // namespace na
