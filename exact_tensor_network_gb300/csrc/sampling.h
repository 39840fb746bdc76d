// Outcomes drawn from rows: the handle, the kernels' arguments and their
// launchers.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/tn_sampling.h"
#include "outcomes.h"

namespace tn {

// A piece of a row: what one warp reads in two steps.  Its weights' sum is kept.
constexpr int kPieceVecs = 64;
constexpr int kDrawThreads = 256;       // CTA of the kernels
constexpr int kDrawWarps = kDrawThreads / 32;
// Rows are cut into segments of a multiple of kDrawWarps pieces, one CTA each,
// until that many CTAs run (as many as fit the SMs at once).
constexpr int64_t kDrawTarget = 4 * kOutSms;
// Rows of at most this many vectors (8 KiB) stay in registers from end to end (bf16, without filters
// and with top_p: 1024 x 4088 24 and 53 us, in segments 1024 x 4104 38 and 116; 8000 rows 148
// and 386, 220 and 798).
constexpr int kRowVecs = 512;
// Bins by which filters narrow down to the entry where they cut, the entries of
// their range that are looked at one by one, and the rows from which there is a second level of bins.
constexpr int kBins = 4096;
constexpr int kSorted = 2048;
constexpr int64_t kLongRow = 1 << 18;
// Draws of a row that the CTA makes which finishes the row's sums (64 x 50000 bf16: 8 draws 37 us by
// those CTAs, 40 by a kernel of their own; 16 draws 51 and 39).
constexpr int64_t kFewDraws = kDrawWarps;

struct RowState;
struct RowBins;

struct SampleArgs {
    OutRows r;
    tn_filters f;
    const void *u;
    int64_t *ids;
    float *logp;
    int64_t *kept;
    int64_t draws;
    int32_t wide;
    bool filtered;          // top_k or top_p of a row may leave less than all
    bool powers;            // beta of a row may be other than 1
    int64_t pieces;         // of a row
    int64_t segs, seg_pieces;
    uint64_t *masses;       // [rows][pieces]
    uint32_t *ties;         // [rows][pieces] equal entries where a filter cuts through many
    // of rows in segments: state [rows]; partial results [rows][segs] of
    // segments, first maxima with rough sums, then sums and counts, and sums of all
    // entries; and, of several segments, bins [rows] and lists [rows][kSorted]
    RowState *state;
    ulonglong2 *partials;
    uint64_t *alls;
    RowBins *bins;
    uint64_t *lists;
};

struct Sampler {
    int32_t type = 0;
    int64_t cols = 0, max_rows = 0;
    float scale = 1.f;
    uint64_t ws_bytes = 0, clear_bytes = 0;
    uint64_t state_off = 0, bins_off = 0, partial_off = 0, rest_off = 0, list_off = 0, mass_off = 0, tie_off = 0;
    char *ws = nullptr;
    char error[256] = {0};
};

// of a row
int64_t state_bytes();
int64_t bins_bytes();

template <int TYPE>
cudaError_t sample_of(const SampleArgs &a, cudaStream_t stream);

}  // namespace tn

struct tn_sampler_s {
    tn::Sampler s;
};
