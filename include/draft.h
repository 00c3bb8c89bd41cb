/*
 * draft.h -- C ABI of libw12.so's verification of drafted tokens, the end of a
 * verify step of speculative decoding, for AMD MI355X (gfx950).
 *
 * Conventions: those of mx4.h (device pointers owned by the caller, work
 * enqueued on `stream`, arguments checked on the host before any launch, the
 * w12_status_t values returned, nothing allocated or kept, no synchronisation,
 * the same bits for the same call).
 */
#ifndef DRAFT_H
#define DRAFT_H

#include <stddef.h>
#include <stdint.h>

#include "w12.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DRAFT_MAX_D 1023        /* drafted tokens a sequence */

/* Static, never-NULL description of a status code, in the terms of the calls
 * below. */
const char *draft_status_string(int status);

/*
 * draft_verify -- which drafted tokens of each sequence b the target's
 * probabilities accept, and the token that follows them.  With n = lengths[b]
 * drafted tokens x_i = drafts[b, i], the target's logits l_i = logits[b, i] of
 * rows i = 0 .. n, and tau = temperature[b] (1 without one):
 *   p_i      = softmax(l_i / tau);
 *   q_i      = draft_probs[b, i], what x_i was drawn from (without draft_probs:
 *              x_i itself with probability 1);
 *   x_i is accepted if all before it are and
 *              uniforms[b, i] * q_i(x_i) < p_i(x_i);
 *   a        = the accepted tokens; the one behind them is drawn from
 *              max(0, p_a - q_a) if x_a was refused (from p_a where that is 0
 *              everywhere), from p_n if a = n: the first word v whose running
 *              sum of weights, in the order of the words, exceeds
 *              uniforms[b, D] times their whole sum, or the last of positive
 *              weight if rounding leaves none.
 * tau <= 0 (or NaN) is greedy: x_i is accepted if it is l_i's largest logit's
 * word (the lowest of a tie), and the token behind is that word of row a.
 *   tokens[b, .]  = the a accepted tokens, the one behind them, then -1;
 *   accepted[b]   = a.
 * Probabilities, their sums and the running sums are held in 64 bits; a word
 * of less than 2^-1000 of its row's largest probability counts as 0.
 * A row that holds a NaN or +inf, or nothing but -inf, has no distribution: its
 * draft is refused, and the token drawn from it is -1.  A draft outside
 * 0 .. V-1 is refused, and what is drawn then is as if q were q_a with nothing
 * taken off for it (with draft_probs: max(0, p_a - q_a); without: p_a).
 *   logits      : device [B, D + 1, V], BF16 bits or fp32 as logits_type (a
 *                 w12_out_t) says, strides ldb and ldd elements between
 *                 sequences and rows, words contiguous, aligned to its type.
 *                 Rows past lengths[b] are not read.
 *   drafts      : device [B, D] contiguous, int32 (drafts_i64 = 0) or int64.
 *   uniforms    : device fp32 [B, D + 1] contiguous, in [0, 1).
 *   draft_probs : device [B, D, V], BF16 bits or fp32 as probs_type says, not
 *                 negative, strides pdb and pdd elements; or NULL.
 *   lengths     : device int32 [B], taken as 0 below 0 and as D above D; or
 *                 NULL: all D.
 *   temperature : device fp32 [B]; or NULL.
 *   tokens      : device int32 output [B, D + 1].
 *   accepted    : device int32 output [B].
 *   workspace   : draft_workspace_bytes(B, D, V) bytes, 256-byte aligned.
 * 0 <= D <= DRAFT_MAX_D, 1 <= V <= 2^30, B * (D + 1) <= 2^24 and
 * B * (D + 1) * V <= 2^40.  B = 0 launches nothing.
 * Errors: W12_ERR_NULL, W12_ERR_SHAPE, W12_ERR_DTYPE, W12_ERR_ALIGN,
 *         W12_ERR_UNSUPPORTED (D over its limit), W12_ERR_WORKSPACE,
 *         W12_ERR_HIP.
 */
int draft_verify(const void *logits, int logits_type, int64_t B, int64_t D, int64_t V,
                 int64_t ldb, int64_t ldd, const void *drafts, int drafts_i64,
                 const float *uniforms, const void *draft_probs, int probs_type, int64_t pdb,
                 int64_t pdd, const int32_t *lengths, const float *temperature, int32_t *tokens,
                 int32_t *accepted, void *workspace, size_t workspace_bytes, void *stream);
int draft_workspace_bytes(int64_t B, int64_t D, int64_t V, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* DRAFT_H */
