// Drawing outcomes from rows of fp32 logits.
#include "sampling.cuh"

namespace tn {

template cudaError_t sample_of<TN_TYPE_F32>(const SampleArgs &, cudaStream_t);

}  // namespace tn
