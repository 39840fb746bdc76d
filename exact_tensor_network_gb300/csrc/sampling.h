// Outcomes drawn from rows: the handle, the kernels' arguments and their
// launchers.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/tn_sampling.h"
#include "outcomes.h"

namespace tn {

// A piece of a row: what one warp reads in four steps.  Its weights' sum is kept.
constexpr int kPieceVecs = 128;
constexpr int kRowThreads = 256;        // CTA of a row

struct SampleArgs {
    OutRows r;
    tn_filters f;
    const void *u;
    int64_t *ids;
    float *logp;
    int64_t *kept;
    int64_t draws;
    int32_t wide;
    int64_t pieces;         // of a row
    uint64_t *masses;       // [rows][pieces]
};

struct Sampler {
    int32_t type = 0;
    int64_t cols = 0, max_rows = 0;
    float scale = 1.f;
    uint64_t ws_bytes = 0, mass_off = 0;
    char *ws = nullptr;
    char error[256] = {0};
};

template <int TYPE>
cudaError_t sample_of(const SampleArgs &a, cudaStream_t stream);

}  // namespace tn

struct tn_sampler_s {
    tn::Sampler s;
};
