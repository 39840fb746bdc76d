/*
 * tn_outcomes.h: operators on outcome distributions.
 *
 * A contraction with open modes (tn_execute) answers with a batch of rows of
 * amplitudes over the outcomes of its open qubits; a network that is the head
 * of a model answers with rows of real logits.  These calls turn such rows
 * into what is asked of them next: log probabilities of given outcomes, the
 * entropy and the most likely outcomes of a row (tn_outcomes_score), the loss
 * against a teacher that is known by its top logits (tn_outcomes_distill), and
 * the gradients of both.
 *
 * Definitions.  A row has `cols` entries.  The logit z of an entry is the real
 * entry itself, or ln w with w = re^2 + im^2 for an amplitude (the two squares
 * and the sum each rounded to fp32: w must lie in fp32's range; one below 2^-126
 * has fewer digits, and may count as 0 in a sum at other scales than 1).
 *   - An entry is absent if its mask byte is 0 or z = -inf (w = 0).  What lies
 *     in masked places is never used (NaN and infinities included).
 *   - log Z = ln sum exp(scale z) over the present entries, log p = scale z -
 *     log Z, entropy H = - sum p log p.  scale is the inverse temperature.
 *     log p, losses and training steps are taken from differences of logits, so
 *     they hold where log Z rounds by more than ln V (large logits, as where a
 *     mask was written as one) or, scale z being beyond fp32, is infinite.  The
 *     gradient calls that are given log Z have its rounding: p to about
 *     2^-23 |log Z|.
 *   - Alternatives: the present entries of largest z (largest w for
 *     amplitudes), ties to the lowest index; id -1 and log p -inf past the
 *     number of present entries.
 *   - A row without present entries has log Z = -inf, H = 0, log p = -inf, no
 *     alternatives, loss 0 and gradient 0.
 *   - A present NaN or +inf leaves the row without a distribution: its fp32
 *     outputs are NaN, its alternatives' ids -1.
 *   - Ids are int64.  -1 means "none" (log p 0, no gradient, not part of the
 *     teacher).  An id below -1 or not below cols reads nothing: its log p (or
 *     its row's loss) is NaN, it has no gradient, and tn_outcomes_check
 *     reports TN_EDEVICE.
 *
 * Conventions are those of tn.h: no call throws, every failure is a tn_status,
 * the library allocates no device memory, work is enqueued on the caller's
 * stream and the calls return at once.  All arithmetic is fp32 whatever the
 * rows' type; gradients are rounded to it once.  Results do not depend on
 * timing (no floating-point atomics).  A handle belongs to one host thread and
 * one stream at a time (its workspace carries partial sums between CTAs).
 * Every call can be captured into a CUDA graph.
 */
#ifndef TN_GB300_OUTCOMES_H
#define TN_GB300_OUTCOMES_H

#include "tn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Entry types. */
enum {
    TN_TYPE_C64 = 0,  /* amplitudes: interleaved fp32 (re, im), as tn_execute writes */
    TN_TYPE_F32 = 1,  /* real logits */
    TN_TYPE_BF16 = 2,
    TN_TYPE_F16 = 3
};

enum {
    TN_OUTCOMES_MAX_TOP = 128,   /* alternatives per row */
    TN_OUTCOMES_MAX_IDS = 256    /* given outcomes or teacher's outcomes per row */
};

/* A batch of rows in device memory.  Strides are in entries; entry (r, v) lies
 * at data[r row_stride + v col_stride].  col_stride 1 is the fast layout.
 * data is aligned to its entry type (8 bytes for TN_TYPE_C64).  mask: one byte
 * per entry with its own strides (0 repeats a row or a column), or NULL. */
typedef struct tn_rows {
    const void *data;
    int64_t rows;
    int64_t row_stride, col_stride;
    const uint8_t *mask;
    int64_t mask_row_stride, mask_col_stride;
} tn_rows;

/* The teacher of tn_outcomes_distill*: `count` outcomes per row (1 ..
 * TN_OUTCOMES_MAX_IDS), contiguous.  q = softmax(scale * logits) over the
 * outcomes of the row that are neither -1 nor masked in the student's row.
 * Log probabilities are logits too (scale 1 keeps them). */
typedef struct tn_teacher {
    const int64_t *ids;     /* [rows, count] */
    const void *logits;     /* [rows, count] of `type` */
    int32_t type;           /* TN_TYPE_F32, TN_TYPE_BF16 or TN_TYPE_F16 */
    int32_t count;
    float scale;
} tn_teacher;

typedef struct tn_outcomes_s tn_outcomes_t;

/*
 * Make a handle for rows of `cols` entries of `type`, at most `max_rows` rows
 * and `max_top` alternatives (0 .. TN_OUTCOMES_MAX_TOP) per call, at inverse
 * temperature `scale` (2^-40 .. 2^40).  Host only.  Errors: TN_EINVAL (a value
 * outside its range; see tn_outcomes_last_error(NULL)), TN_EOVERFLOW.
 */
TN_API tn_status tn_outcomes_create(int32_t type, int64_t cols, int64_t max_rows, int32_t max_top,
                                    float scale, tn_outcomes_t **out);

/* Release a handle (NULL is ignored).  Does not free the workspace. */
TN_API void tn_outcomes_destroy(tn_outcomes_t *h);

/* Device workspace of the handle, in bytes. */
TN_API tn_status tn_outcomes_workspace_bytes(const tn_outcomes_t *h, uint64_t *bytes);

/* Bind memory of the current device, on which all calls on the handle have to
 * be made (256-byte aligned, at least that large, owned by the caller and left
 * alone by everyone else while bound).  Clears its status word (synchronous,
 * so not while a stream is captured).  Errors: TN_EINVAL, TN_ENOMEM (too small), TN_ECUDA. */
TN_API tn_status tn_outcomes_set_workspace(tn_outcomes_t *h, void *dev_ptr, uint64_t bytes);

/*
 * Scores of every row.
 *   given      [rows, n_given] outcomes (n_given 0 .. TN_OUTCOMES_MAX_IDS)
 *   logp       [rows, n_given] their log probabilities
 *   logz       [rows]          log Z
 *   entropy    [rows]          H
 *   top_ids    [rows, n_top]   the n_top <= max_top most likely outcomes
 *   top_logp   [rows, n_top]   and their log probabilities, in descending order
 * All contiguous; given, logp (with n_given = 0) and top_ids, top_logp (with
 * n_top = 0) may be NULL.  The rows are read once, but for the few pieces of them
 * that hold the alternatives.
 * Errors of this and the calls below: TN_EINVAL (arguments), TN_ENOMEM (no
 * workspace), TN_ECUDA (launch).
 */
TN_API tn_status tn_outcomes_score(tn_outcomes_t *h, const tn_rows *rows, const int64_t *given,
                                   int32_t n_given, float *logp, float *logz, float *entropy,
                                   int32_t n_top, int64_t *top_ids, float *top_logp,
                                   tn_stream_t stream);

/*
 * Gradient of L through tn_outcomes_score's logp and entropy:
 *   dL/dz_v = scale (sum_j g_j [given_j = v] - p_v (sum_j g_j + h (log p_v + H)))
 * with g = g_logp [rows, n_given] (given outcomes that are absent or -1 carry
 * none; the same outcome given twice adds up) and h = g_entropy [rows] (NULL:
 * none).  logz and entropy are those of the forward call (entropy may be NULL
 * without g_entropy).  grad: entry (r, v) at grad[r grad_row_stride + v
 * grad_col_stride], in the rows' type; every entry is written, 0 where absent.
 * For amplitudes grad = dL/dRe + i dL/dIm = 2 a / |a|^2 dL/dz.
 * grad may not overlap the rows.  The alternatives' log probabilities are
 * differentiated by giving their ids.  For TN_TYPE_F32 and TN_TYPE_F16 a p below
 * 2^-126 may count as 0, here and in the other gradients.
 */
TN_API tn_status tn_outcomes_score_grad(tn_outcomes_t *h, const tn_rows *rows, const int64_t *given,
                                        int32_t n_given, const float *logz, const float *entropy,
                                        const float *g_logp, const float *g_entropy, void *grad,
                                        int64_t grad_row_stride, int64_t grad_col_stride,
                                        tn_stream_t stream);

/*
 * Distance of every row from a teacher: loss[r] = sum_j q_j (log q_j -
 * log p of its outcome j).  +inf where the teacher expects an outcome whose
 * unmasked logit is -inf; 0 where the row is empty or the teacher has nothing
 * left.  logz: [rows], kept for the gradient.
 */
TN_API tn_status tn_outcomes_distill(tn_outcomes_t *h, const tn_rows *rows,
                                     const tn_teacher *teacher, float *loss, float *logz,
                                     tn_stream_t stream);

/* Its gradient: dL/dz_v = g_loss[r] scale (p_v - sum_j q_j [ids_j = v]), laid
 * out as in tn_outcomes_score_grad. */
TN_API tn_status tn_outcomes_distill_grad(tn_outcomes_t *h, const tn_rows *rows,
                                          const tn_teacher *teacher, const float *logz,
                                          const float *g_loss, void *grad, int64_t grad_row_stride,
                                          int64_t grad_col_stride, tn_stream_t stream);

/* Loss and gradient together, where g_loss is known beforehand (a mean over
 * the batch: 1 / rows): the results of the two calls above, but for a rounding,
 * and without that of log Z (see the definitions) unless the rows are long and
 * read twice. */
TN_API tn_status tn_outcomes_distill_step(tn_outcomes_t *h, const tn_rows *rows,
                                          const tn_teacher *teacher, const float *g_loss,
                                          float *loss, float *logz, void *grad,
                                          int64_t grad_row_stride, int64_t grad_col_stride,
                                          tn_stream_t stream);

/* After the stream has been synchronised: read and clear the handle's device
 * status word.  TN_OK, or TN_EDEVICE (an id outside [-1, cols)). */
TN_API tn_status tn_outcomes_check(tn_outcomes_t *h);

/* Text of the last failure on this handle; with h == NULL, of the last failed
 * tn_outcomes_create() on this thread. */
TN_API const char *tn_outcomes_last_error(const tn_outcomes_t *h);

#ifdef __cplusplus
}
#endif

#endif /* TN_GB300_OUTCOMES_H */
