/*
 * mx4_route.h -- C ABI of libw12.so's routing of tokens to experts, and of the
 * expert layer of mx4.h on such a routing, for AMD MI355X (gfx950).
 *
 * Conventions: those of mx4.h.
 */
#ifndef MX4_ROUTE_H
#define MX4_ROUTE_H

#include <stddef.h>
#include <stdint.h>

#include "w12.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
    MX4_SCORE_SOFTMAX = 0,      /* s(t, e) = exp(l[t, e]) / sum over all e' of exp(l[t, e']) */
    MX4_SCORE_SIGMOID = 1       /* s(t, e) = 1 / (1 + exp(-l[t, e])) */
};

#define MX4_MAX_ROUTE_T ((int64_t)1 << 24)      /* tokens of one mx4_route call */
#define MX4_MAX_GROUPS 64                       /* its groups of experts */

/*
 * mx4_route -- each token's experts and their shares:
 *   rank(t, e)  = s(t, e) + bias[e] with a bias, else the logit l[t, e] itself
 *                 (the order of the scores);
 *   group       = E / groups consecutive experts.  With kept_groups < groups
 *                 only the kept_groups groups with the largest value count:
 *                 group_terms = 1: the largest rank in the group; 2: the sum of
 *                 its two largest s(t, e) + bias[e] (of its only one, if it has
 *                 no other);
 *   S(t)        = the top_k experts of the counting groups with the largest
 *                 rank; every tie goes to the lowest index;
 *   share       = scale * s(t, e) / sum over S(t) of s(t, .)  (renormalize != 0;
 *                 0 where that sum is 0), or scale * s(t, e).
 * Scores, ranks and sums are held in 64 bits, shares are rounded once to fp32;
 * an exponential is off by less than 2.8e-14 of itself (exp(0) is 1), and below
 * exp(-707) counts as 0.
 * An expert whose logit or whose bias is -inf is in no S(t) and adds nothing to
 * its group's value; a token with fewer than top_k others gets -1 and share 0
 * in the places left.
 * A NaN rank, a logit's or a bias's, is above all others, a group's value NaN
 * that it goes into (or, of two terms, a NaN score) above all other groups',
 * and ties go to the lowest as elsewhere.  A NaN logit makes its own share NaN,
 * and under softmax or renormalisation all of its token's.  Under softmax a
 * token with a logit of NaN or +inf has no scores: all its shares are NaN, and
 * where scores decide all its ranks (with a bias) or all its groups' values (of
 * two terms) are alike, so that the lowest experts or groups are taken that have
 * or hold a logit and a bias above -inf.
 *   logits  : device [T, E], BF16 bits or fp32 as logits_type (a w12_out_t)
 *             says, row stride ldl >= E elements, aligned to its type.
 *   bias    : device fp32 [E], or NULL.
 *   experts : device int32 output [T, top_k], in the order of their rank.
 *   shares  : device fp32 output [T, top_k].
 * E <= MX4_MAX_E, top_k <= MX4_MAX_TOP_K (mx4.h) and top_k <= E;
 * groups <= MX4_MAX_GROUPS, E % groups == 0, 1 <= kept_groups <= groups,
 * group_terms 1 or 2.
 * Errors: W12_ERR_NULL, W12_ERR_SHAPE, W12_ERR_DTYPE (logits_type or score),
 *         W12_ERR_ALIGN, W12_ERR_UNSUPPORTED (T, E, groups or top_k over its
 *         limit), W12_ERR_HIP.
 */
int mx4_route(const void *logits, int logits_type, int64_t T, int64_t E, int64_t ldl,
              const float *bias, int score, int64_t groups, int64_t kept_groups, int group_terms,
              int64_t top_k, int renormalize, float scale, int32_t *experts, float *shares,
              void *stream);

/*
 * mx4_moe_routed -- mx4_moe (mx4.h) with the choice given:
 *   y[t] = sum over j of shares[t, j] * D_e h(t, e),  e = experts[t, j].
 * An entry of experts outside 0 .. E-1 counts for nothing, whatever its share;
 * an expert that a token names twice counts with both shares.
 *   experts, shares : device int32 and fp32 [T, top_k], contiguous.
 * The rest, limits and errors are mx4_moe's, the workspace too
 * (mx4_moe_workspace_bytes).
 */
int mx4_moe_routed(const uint16_t *x, int64_t T, int64_t ldx, const int32_t *experts,
                   const float *shares, const void *w13_codes, const void *w13_scales,
                   const void *w2_codes, const void *w2_scales, int64_t H, int64_t I, int64_t E,
                   int64_t top_k, void *y, int64_t ldy, int y_type, void *workspace,
                   size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MX4_ROUTE_H */
