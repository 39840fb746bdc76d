// Drawing outcomes from rows of fp16 logits.
#include "sampling.cuh"

namespace tn {

template cudaError_t sample_of<TN_TYPE_F16>(const SampleArgs &, cudaStream_t);

}  // namespace tn
