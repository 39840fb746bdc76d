// Drawing outcomes from rows of amplitudes.
#include "sampling.cuh"

namespace tn {

int64_t state_bytes() { return sizeof(RowState); }
int64_t bins_bytes() { return sizeof(RowBins); }

template cudaError_t sample_of<TN_TYPE_C64>(const SampleArgs &, cudaStream_t);

}  // namespace tn
