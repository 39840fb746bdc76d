// The outcome operators' kernels for f16 logits.
#include "outcomes_step.cuh"

namespace tn {

template cudaError_t outcomes_forward_of<TN_TYPE_F16>(const OutForward &, bool, cudaStream_t);
template cudaError_t outcomes_grad_of<TN_TYPE_F16>(const OutGrad &, bool, cudaStream_t);
template cudaError_t outcomes_step_of<TN_TYPE_F16>(const OutStep &, bool, cudaStream_t);

}  // namespace tn
