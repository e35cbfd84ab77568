// Gated feed-forward product on CUDA cores and sums of the products' runs, bf16 (see na_glu_fma.cuh).
#include "na_glu_fma.cuh"

namespace na {
namespace glu {
template na_status launch_fma<__nv_bfloat16>(const GluParams&, Product, const FmaTile&, cudaStream_t);
template na_status launch_sum<__nv_bfloat16>(const float*, int, long long, long long, void*, void*, cudaStream_t);
}  // namespace glu
}  // namespace na
