/*
 * tq_sample.h -- the end of a decode step: a token for each row of logits.
 * tq.h's conventions hold: device pointers owned by the caller, work enqueued on
 * `stream`, arguments checked before anything is launched, no allocation, no
 * synchronisation, contiguous row-major arrays, outputs that overlap no input.
 * (The source pages have no counterpart to this header.)
 */
#ifndef TQ_SAMPLE_H
#define TQ_SAMPLE_H

#include "tq.h"
#include "tq_moe.h" /* tq_dtype */

#ifdef __cplusplus
extern "C" {
#endif

#define TQ_SAMPLE_MAX_VOCAB (1 << 20)
#define TQ_SAMPLE_MAX_ROWS (1 << 20)

/* Draw a token for each of m rows of logits [m][vocab] of logits_type
 * (tq_dtype).  An entry that is NaN or -infinity is no candidate, +infinity
 * counts as the largest finite number.  For a row, its candidates in the order of
 * descending logits, ties to the lowest index:
 *   weights  w_i = exp((l_i - l_max) / temperature)
 *   top-k    the first top_k stay
 *   min-p    of them those with w_i >= min_p, and the first always
 *   top-p    of them the shortest run from the first on whose sum is at least
 *            top_p times the sum of all of them, and the first always
 *   draw     the lowest index i at which the sum of what stayed, over the
 *            indices up to i, exceeds  uniform * (the sum of what stayed)
 * ids[r] = i; probs[r] (may be NULL) = w_i / (the sum of what stayed).  A row
 * without candidates has -1 and 0.
 * Per-row settings, each [m] or NULL for none of it:
 *   temperature fp32: below 2^-99 (0, negative) or NaN: the first of the order,
 *     with probability 1 (the row's other settings are not looked at); NULL: 1;
 *     +infinity: equal weights
 *   top_k int32: <= 0 or more than there are: all
 *   top_p fp32: >= 1 or NaN: all; <= 0: the first
 *   min_p fp32: <= 0 or NaN: all; > 1 counts as 1
 * uniform: fp32 [m], in [0, 1); NaN or below 0 counts as 0, and from 1 on the last
 * index that stayed with a weight above 0 is drawn (below 2^-43 it rounds to 0).
 * Weights are whole multiples of 2^-42, each off by up to 2^-43 and about 2^-30 of
 * itself, and sums of them are exact: the result does not depend on how a row is split
 * over threads.  A sum of n weights is off by up to n * 2^-43 and 2^-30 of itself (2^-23 of
 * it where all of the largest vocabulary is a tail of weights near 2^-42), and the result
 * differs from that of real arithmetic only where a sum comes that near to a border;
 * a probability is off by what its weight and the sum are, and by its rounding.  A row's
 * results do not depend on the other rows.
 * logits aligned to their type; the other arrays 4-byte aligned;
 * 1 <= vocab <= TQ_SAMPLE_MAX_VOCAB, 1 <= m <= TQ_SAMPLE_MAX_ROWS. */
tq_status tq_sample(const void *logits, int32_t logits_type, int32_t m, int32_t vocab,
                    const float *temperature, const int32_t *top_k, const float *top_p,
                    const float *min_p, const float *uniform, int32_t *ids, float *probs,
                    tq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TQ_SAMPLE_H */
