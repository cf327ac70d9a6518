/*
 * spear_sample.h - drawing a step's tokens from its logits.
 *
 * Conventions are spear.h's: device pointers owned by the caller, every call
 * asynchronous on the stream it is given, no device memory allocated and
 * nothing copied between host and device, arguments validated on the host
 * before anything is launched, spear_last_error() for the detail.  What only
 * the device can see (the values of the per-row arrays) never makes the
 * kernels read or write outside the arrays described here.
 */
#ifndef SPEAR_SAMPLE_H
#define SPEAR_SAMPLE_H

#include "spear_mx.h" /* SPEAR_F32 */

#ifdef __cplusplus
extern "C" {
#endif

/*
 * One token per row of logits, from the row's random number.
 *
 * A row's tokens are taken in descending order of their logits l, ties by the
 * lowest index, with weights w = exp((l - max) / T).  Kept are those that are
 *   - among the first k,
 *   - and whose predecessors weigh less than p times the weight of the first
 *     k together (the first token always is),
 *   - and whose weight is at least min_p (the largest weight is 1).
 * The token is the first whose cumulative weight is above u times the weight
 * of all that is kept; its logprob is the logarithm of its own share of it.
 * Weights are rounded to 32 places and summed in 64 bits, in an order that does
 * not depend on timing.
 *
 * A logit of -infinity or NaN is never drawn.  Where a row has logits of
 * +infinity, those alone are drawn, all with weight 1.  A row with nothing to
 * draw gives token -1 and logprob -infinity.  Tokens that weigh less than
 * e^-64 count among the first k, but their own weight counts as 0.
 *
 *   logits       [rows] of vocab values, stride elements apart (>= 0), of
 *                dtype SPEAR_F16, SPEAR_BF16 or SPEAR_F32.
 *   u            [rows]: in [0, 1).  Below: as 0 (NaN too); from 1 on: the last token kept (of
 *                those that weigh e^-64 or more).
 *   temperature  [rows] or NULL (1): T.  Not above 0: the first token is taken, whatever k, p,
 *                min_p and u are.
 *   top_k        [rows] or NULL (0): k.  Not above 0: no limit.
 *   top_p        [rows] or NULL (1): p.  Not below 1: no limit.
 *   min_p        [rows] or NULL (0).  Not above 0: no limit; above 1: as 1.
 *   tokens       [rows]: indices into the row.
 *   logprobs     [rows] or NULL.
 * rows 0..2^20, vocab 1..2^18.
 */
typedef struct spear_sample_args {
  const void *logits;
  int32_t dtype, rows, vocab;
  int64_t stride;
  const float *u, *temperature;
  const int32_t *top_k;
  const float *top_p, *min_p;
  int32_t *tokens;
  float *logprobs;
} spear_sample_args_t;

/*
 * Workspace bytes that spear_sample needs for at most these sizes; 0 when one
 * is invalid.  256-byte aligned, its first SPEAR_SAMPLE_HEADER_BYTES ZEROED
 * ONCE before its first use, left ready by every call.  It overlaps nothing
 * that the call reads or writes; calls that may overlap need different ones.
 */
#define SPEAR_SAMPLE_HEADER_BYTES 16384
size_t spear_sample_workspace_bytes(int32_t rows, int32_t vocab);
spear_status_t spear_sample(const spear_sample_args_t *args, void *workspace,
                            size_t workspace_bytes, spear_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEAR_SAMPLE_H */
