// Residual add between norms, forward, fp32 (see na_add_impl.cuh).
#include "na_add_impl.cuh"

namespace na {
namespace add {
template na_status launch_add<float, false>(const AddParams&, const AddPlan&, cudaStream_t);
}  // namespace add
}  // namespace na
