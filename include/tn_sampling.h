/*
 * tn_sampling.h: outcomes drawn from rows by given random numbers.
 *
 * Rows are those of tn_outcomes.h: amplitudes over the outcomes of a
 * contraction's open qubits (drawn by the Born rule), or a model's logits.
 *
 * Definitions.  Logits z, absent entries and rows without a distribution are
 * those of tn_outcomes.h.
 *   - With beta = scale / temperature (one fp32 division; a quotient beyond fp32
 *     counts as the largest number) a present entry's weight is exp(beta z), relative to
 *     the largest (of which logits that are further from it than fp32 reaches count as
 *     that far).
 *   - Three filters follow each other.  top_k: the entries of largest z (largest
 *     w for amplitudes), ties to the lowest index.  top_p: of those, in that
 *     order, the fewest whose weight is at least top_p times that of all of
 *     them, one at least.  min_p: of those, the ones of weight >= min_p times the largest.
 *     top_k <= 0, top_p >= 1 and min_p <= 0 leave all.
 *   - A temperature of 0 is greedy: of all entries, the largest is left, of the lowest index
 *     among equals.
 *   - The outcome drawn with a random number u in [0, 1) is the first entry left, in the order
 *     of indices, for which the weights of the entries left up to and with it sum to
 *     more than u times that of all left.
 *   - log p of a draw is that of its outcome among the entries left; `kept` is their
 *     number.
 *   - A row without present entries has outcome -1, log p -inf and kept 0; a row
 *     without a distribution, or one with an invalid parameter, outcome -1, log p NaN and
 *     kept 0.  A draw with an invalid u has outcome -1 and log p NaN.
 * Weights are computed to some 2^-43 of the largest (those of amplitudes at a beta other than
 * 1 and up to 2 to 2^-40) and summed as 64-bit integers, so that an outcome is that of the
 * definition but where u (or top_p) lies that near to a border between two.  Results do not
 * depend on timing.
 *
 * Invalid parameters: a temperature that is negative or no finite number, a NaN top_p or
 * min_p, a min_p above 1, a u outside [0, 1).  tn_sampler_check reports them.
 *
 * Conventions are those of tn_outcomes.h: no call throws, the library
 * allocates no device memory, work is enqueued on the caller's stream, a handle
 * belongs to one host thread and one stream at a time, every call can be
 * captured into a CUDA graph.
 */
#ifndef TN_GB300_SAMPLING_H
#define TN_GB300_SAMPLING_H

#include "tn_outcomes.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Parameters of the draws: one number for all rows, or where the pointer is not
 * NULL one for each row (device memory, contiguous). */
typedef struct tn_filters {
    float temperature, top_p, min_p;
    int32_t top_k;
    const float *temperatures, *top_ps, *min_ps;
    const int32_t *top_ks;
} tn_filters;

typedef struct tn_sampler_s tn_sampler_t;

/*
 * Make a handle for rows of `cols` entries (below 2^31) of `type`, at most `max_rows` rows
 * a call, at inverse temperature `scale` (2^-40 .. 2^40) before any other.
 * Host only.  Errors: TN_EINVAL (a value outside its range; see tn_sampler_last_error(NULL)),
 * TN_EOVERFLOW, TN_ENOMEM.
 */
TN_API tn_status tn_sampler_create(int32_t type, int64_t cols, int64_t max_rows, float scale, tn_sampler_t **out);

/* Release a handle (NULL is ignored).  Does not free the workspace. */
TN_API void tn_sampler_destroy(tn_sampler_t *h);

/* Device workspace of the handle, in bytes. */
TN_API tn_status tn_sampler_workspace_bytes(const tn_sampler_t *h, uint64_t *bytes);

/* Bind memory of the current device, on which all calls on the handle have to be
 * made (256-byte aligned, at least that large, owned by the caller and left alone
 * by everyone else while bound).  Clears what has to be clear (synchronous, so
 * not while a stream is captured).  Errors: TN_EINVAL, TN_ENOMEM (too small), TN_ECUDA. */
TN_API tn_status tn_sampler_set_workspace(tn_sampler_t *h, void *dev_ptr, uint64_t bytes);

/*
 * Draw from every row.
 *   u      [rows, draws] random numbers, of fp32 or (wide != 0) fp64
 *   ids    [rows, draws] outcomes
 *   logp   [rows, draws] their log probabilities
 *   kept   [rows]        the number of entries that the filters leave
 * All contiguous.  filters NULL: temperature 1 and no filter.  draws >= 0; with
 * draws 0, u, ids and logp may be NULL.
 * Errors: TN_EINVAL (arguments), TN_ENOMEM (no workspace), TN_EOVERFLOW, TN_ECUDA (launch).
 */
TN_API tn_status tn_sampler_draw(tn_sampler_t *h, const tn_rows *rows, const tn_filters *filters, const void *u,
                                 int32_t wide, int64_t draws, int64_t *ids, float *logp, int64_t *kept,
                                 tn_stream_t stream);

/* After the stream has been synchronised: read and clear the handle's device
 * status word.  TN_OK, or TN_EDEVICE (an invalid parameter or random number). */
TN_API tn_status tn_sampler_check(tn_sampler_t *h);

/* Text of the last failure on this handle; with h == NULL, of the last failed
 * tn_sampler_create() on this thread. */
TN_API const char *tn_sampler_last_error(const tn_sampler_t *h);

#ifdef __cplusplus
}
#endif

#endif /* TN_GB300_SAMPLING_H */
