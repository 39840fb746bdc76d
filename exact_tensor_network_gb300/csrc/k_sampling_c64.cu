// Drawing outcomes from rows of amplitudes.
#include "sampling.cuh"

namespace tn {

template cudaError_t sample_of<TN_TYPE_C64>(const SampleArgs &, cudaStream_t);

}  // namespace tn
