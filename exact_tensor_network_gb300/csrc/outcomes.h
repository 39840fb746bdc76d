// Operators on outcome distributions: the handle, the kernels' arguments and
// their launchers.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/tn_outcomes.h"
#include "kernels.h"

namespace tn {

constexpr int kOutVecBytes = 16;        // entries are read 16 bytes at a time
constexpr int kOutThreads = 128;        // CTA of the kernels below
constexpr int kOutCtas = 8;             // that many on an SM (64 registers a thread; 6, 10 and 12 were slower)
// Rows of at most this many 16-byte vectors (4 KiB) belong to one warp each:
// a CTA would have no second vector for its threads.
constexpr int kOutWarpVecs = 256;
// Maxima kept for the alternatives, one per 1, 2, 4, .. or 2^kOutChunkLog
// vectors (what a warp reads in one step).
constexpr int kOutKeys = 1024;
constexpr int kOutChunkLog = 7;
constexpr int kOutTree = 2048;          // maxima of a row that one CTA looks at; more form a tree
constexpr int64_t kOutSegVecs = (int64_t)kOutKeys << 5;   // longest segment (512 KiB)

constexpr int kOutSms = 152;
constexpr int64_t kOutTarget = kOutCtas * kOutSms;   // CTAs that fill the GPU

// A first cut for k alternatives keeps up to this many chunks: a bisection
// that may stop anywhere between k and here takes a few steps less.
__host__ __device__ inline int out_most(int k) { return k + k / 8 + 2; }

// Chunks to look at again of a row with a tree; segments and groups of chunks
// on the way to them.
constexpr int kOutList = 1024;
__host__ __device__ inline int out_room(int k) { return 2 * k + 32; }

inline int out_entry_bytes(int32_t type) { return type == TN_TYPE_C64 ? 8 : type == TN_TYPE_F32 ? 4 : 2; }

// How a batch of rows is cut: `segs` segments of `seg_vecs` vectors a row.
struct OutSplit {
    int64_t vecs;       // vectors of the longest row
    int64_t seg_vecs;
    int64_t segs;
    bool warp_rows;     // one warp per row (segs is 1)
};

struct OutRows {
    const char *data;
    int64_t rows, cols, row_stride, col_stride;
    const uint8_t *mask;
    int64_t mask_row_stride, mask_col_stride;
    // log p = scale z - log Z.  c2: weights as powers of two, 2^(c2 z) with
    // c2 = scale log2(e), or (amplitudes) 2^(c2 log2 w) with c2 = scale
    float scale, c2;
    // stands for absent logits in the sums, about -2^126 / max(c2, 1).  Present ones
    // may lie below it where c2 < 1 (the types end near -2^128).
    float floor;
    float lag;          // amplitudes: the quotient by the sums' reference that moves it
    int64_t seg_vecs;
    int64_t segs;
    DevStatus *status;
};

struct OutTeacher {
    const int64_t *ids;
    const void *logits;
    int32_t type, count;
    float scale;
};

// Partial result of a segment: its reference entry and sums (see Sums in
// k_outcomes.cu).
struct OutPartial {
    float z0, s, t;
    int32_t pad;
};

struct OutForward {
    OutRows r;
    // scores
    const int64_t *given;
    float *logp, *logz, *entropy;
    int64_t *top_ids;
    float *top_logp;
    int32_t n_given, n_top;
    // distillation (count 0: scores)
    OutTeacher teacher;
    float *loss;
    // A second kernel finishes the rows (segments, or alternatives of rows of a
    // CTA): partials [rows][segs] and, for alternatives, maxima
    // [rows][segs][seg_chunks] of chunks of 2^chunk_log vectors; with `tree`
    // also supers [rows][segs][33], the maximum of a segment and those of its
    // groups of 32 chunks.
    OutPartial *partials;
    uint32_t *maxima, *supers;
    int32_t finish, tree, seg_chunks, chunk_log;
    // shared memory of a row for the alternatives (see Scratch)
    int32_t key_words, cand_len, group_bytes;
};

struct OutGrad {
    OutRows r;
    const float *logz;
    // scores: ids = given outcomes, g = g_logp
    const int64_t *given;
    const float *entropy, *g_logp, *g_entropy;
    int32_t n_given;
    // distillation (count 0: scores)
    OutTeacher teacher;
    const float *g_loss;
    char *grad;
    int64_t grad_row_stride, grad_col_stride;
};

// Loss and gradient in one kernel: r.segs CTAs of a cluster hold a row,
// r.seg_vecs vectors each.
struct OutStep {
    OutRows r;
    OutTeacher teacher;
    const float *g_loss;
    float *loss, *logz;
    char *grad;
    int64_t grad_row_stride, grad_col_stride;
    bool wide;     // CTAs of twice kStepThreads
};

constexpr int kStepThreads = 128;              // or twice that
// Shared memory of a CTA for its slice and teachers: three CTAs on an SM.
constexpr int64_t kStepSlice = 73 * 1024;
// The most that any step's CTA asks for (four warps' rows and teachers).
constexpr int64_t kStepMemory = 4 * (16 * 1024 + 9 * 1024);
constexpr int kStepCluster = 8;

// Shared memory of a row's teacher (see Teacher): id, q, log q and value of
// each outcome, and a flag.
__host__ __device__ inline int teacher_bytes(int count) { return (count * 20 + 16 + 15) / 16 * 16; }

// What finds repeated ids (see Repeats): two tables, of four places an id or
// more, and a mark for each.
__host__ __device__ inline int repeat_slots(int count) {
    int s = 32;
    while (s < 4 * count) s *= 2;
    return s;
}
__host__ __device__ inline int repeat_marks(int count) { return (count + 15) / 16 * 16; }
__host__ __device__ inline int repeat_bytes(int count) { return 2 * repeat_slots(count) + repeat_marks(count); }
// and of rows of one warp, a sum for each id
__host__ __device__ inline int repeat_sums(int count) { return (count * 4 + 15) / 16 * 16; }
// Shared memory of a training step's CTA besides its slices: two rows'
// teachers and marks, one pair of tables.
__host__ __device__ inline int step_lists(int count) {
    return 2 * (teacher_bytes(count) + repeat_marks(count)) + 2 * repeat_slots(count);
}

struct Outcomes {
    int32_t type = 0;
    int64_t cols = 0, max_rows = 0;
    int32_t max_top = 0;
    float scale = 1.f;
    uint64_t ws_bytes = 0;
    uint64_t partial_off = 0, maxima_off = 0, super_off = 0;
    char *ws = nullptr;
    char error[256] = {0};
};

// aligned: every row starts at a 16-byte boundary.
OutSplit out_split(int32_t type, int64_t cols, int64_t rows, bool aligned, int64_t warp_vecs);
// Launchers, instantiated by k_outcomes_<type>.cu.
template <int TYPE>
cudaError_t outcomes_forward_of(const OutForward &a, bool warp_rows, cudaStream_t stream);
template <int TYPE>
cudaError_t outcomes_grad_of(const OutGrad &a, bool warp_rows, cudaStream_t stream);
template <int TYPE>
cudaError_t outcomes_step_of(const OutStep &a, bool warp_rows, cudaStream_t stream);

}  // namespace tn

struct tn_outcomes_s {
    tn::Outcomes o;
};
