/*
 * tn_block8.h: matrices in 8 bits with a scale for each block of 128, and
 * their products.
 *
 * A contraction's nodes are products of row-major [m, k] and [n, k] matrices
 * (tn.h); a model's head, whose rows of logits the operators of tn_outcomes.h
 * and tn_sampling.h work on, is one with the weights as its second operand.
 * These calls keep such real operands in 8 bits.
 *
 * Definitions.
 *   - A block is 128 consecutive entries of a row (the row's last may be
 *     shorter), or of 128 consecutive rows (block_rows 128: 128 x 128 entries).
 *   - Its scale s is the smallest power of two from 2^-126 on with
 *     max |x| <= 448 s, or 1 if all its entries are 0.  A block that holds a
 *     NaN or an infinity has the scale NaN and codes 0, so that what is
 *     computed from it is NaN.
 *   - A code is x / s rounded to e4m3 (4 exponent bits, 3 of mantissa, no
 *     infinities; to nearest, ties to even) and stands for code * s.
 *   - The product of a [m, k] and b [n, k] is c[i, j] = sum over k of the values
 *     that the codes stand for.  The sums of the codes' products within a block
 *     of k (of up to four, where scales are powers of two) are the tensor core's,
 *     in 32 bits; those over blocks are in fp32, rounded once to the output's
 *     type.  Scales from elsewhere may be any fp32 numbers (powers = 0); those that
 *     tn_block8_quantize makes are powers of two, which products are faster with.
 *
 * Conventions are those of tn.h: no call throws, every failure is a
 * tn_status, no device memory is allocated, work is enqueued on the caller's
 * stream on the current device and the calls return at once.  Results do not
 * depend on timing.  The calls keep nothing (but counts of what went wrong, for
 * tn_block8_check), can be captured into CUDA graphs, and may be made by several host threads
 * and on several streams at once.
 */
#ifndef TN_GB300_BLOCK8_H
#define TN_GB300_BLOCK8_H

#include "tn_outcomes.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { TN_BLOCK8 = 128 };   /* entries of a block along a row */

/* A real matrix of `type` (TN_TYPE_F32, TN_TYPE_BF16 or TN_TYPE_F16): entry
 * (i, j) at data[i row_stride + j col_stride], strides in entries and >= 0;
 * aligned to its entry type.  Either stride 1 is a fast layout. */
typedef struct tn_matrix {
    const void *data;
    int32_t type;
    int64_t rows, cols;
    int64_t row_stride, col_stride;
} tn_matrix;

/* A matrix in 8 bits.  Row i of the codes starts at codes + i row_stride, which
 * is 16-byte aligned (row_stride a multiple of 16, at least cols); what lies
 * between a row's end and the next row is neither read nor written.  The scale of
 * block b of row i is scales[(i / block_rows) scale_stride + b scale_block]; both
 * strides are > 0.  scale_stride 1 is the fast layout of scales of single rows. */
typedef struct tn_block8 {
    uint8_t *codes;
    float *scales;
    int64_t rows, cols;
    int64_t row_stride, scale_stride, scale_block;
    int32_t block_rows;     /* 1 or 128 */
    int32_t powers;         /* nonzero: scales are powers of two (from 2^-126 on) or NaN */
} tn_block8;

/*
 * Codes and scales of x, into `rows` (a matrix of x's shape), into `columns`
 * (of x transposed: its blocks lie along x's columns), or both from one reading of x; the other is
 * NULL.  Both have the same block_rows; with 128 the transposed codes are
 * those of the rows, transposed.  Errors of this and the next call: TN_EINVAL
 * (arguments), TN_EOVERFLOW (sizes), TN_ECUDA (launch).
 */
TN_API tn_status tn_block8_quantize(const tn_matrix *x, const tn_block8 *rows, const tn_block8 *columns,
                                    tn_stream_t stream);

/*
 * out[i, j] = sum_k a[i, k] b[j, k], of `type`, at out[i out_stride + j]
 * (a->rows by b->rows; a->cols = b->cols).  out may not overlap the operands.
 * Without any k (cols 0) the product is 0.
 */
TN_API tn_status tn_block8_product(const tn_block8 *a, const tn_block8 *b, void *out, int32_t type,
                                   int64_t out_stride, tn_stream_t stream);

/* After the device has been synchronised: what the calls on the current device, by any thread,
 * have reported since this host thread's last call of this (or since the process began).
 * TN_OK, TN_ETIMEOUT (a product gave up waiting; its outputs are not valid), or TN_EDEVICE
 * (a scale of a matrix with `powers` is neither a power of two nor NaN; it counted as NaN).
 * One report a call, timeouts first: call until TN_OK.  Other threads are told for themselves. */
TN_API tn_status tn_block8_check(void);

/* Text of this thread's last failed call. */
TN_API const char *tn_block8_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* TN_GB300_BLOCK8_H */
