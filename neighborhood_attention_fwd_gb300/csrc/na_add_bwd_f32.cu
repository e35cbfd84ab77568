// Residual add between norms, backward, fp32 (see na_add_impl.cuh).
#include "na_add_impl.cuh"

namespace na {
namespace add {
template na_status launch_add<float, true>(const AddParams&, const AddPlan&, cudaStream_t);
}  // namespace add
}  // namespace na
