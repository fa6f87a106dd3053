/*
 * sgemm_mi355: routing of tokens to experts, the order of the rows that the
 * experts' products run on, and the weighted return of those rows.
 *
 * Ownership, streams and errors are those of sgemm_mi355.h; element types are
 * those of sgemm_mi355_fp8.h. Matrices without a row stride are dense. `experts` is at
 * least 1 everywhere (else SGEMM_MI355_ERR_DIM).
 */
#ifndef SGEMM_MI355_ROUTE_H
#define SGEMM_MI355_ROUTE_H

#include "sgemm_mi355_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How logits become scores. */
#define SGEMM_MI355_SOFTMAX 0 /* s_i = exp(l_i) / sum_m exp(l_m) */
#define SGEMM_MI355_SIGMOID 1 /* s_i = 1 / (1 + exp(-l_i)) */

#define SGEMM_MI355_MAX_EXPERTS 1024
#define SGEMM_MI355_MAX_CHOICES 32

/*
 * Routing. For each of `tokens` rows of logits (tokens x experts of `type`,
 * row stride ld):
 *   the score s of every expert, and the choice value c_i = s_i + bias_i
 *     (bias: `experts` floats, or null for none; it moves the choice, not the
 *     weights);
 *   with groups > 1, the experts in `groups` equal runs: only the top_groups
 *     groups with the largest sum of their two largest c (their c, where a
 *     group is one expert) stay eligible;
 *   the `choices` eligible experts of largest c, in descending order, to ids
 *     (tokens x choices ints); of equal values the lower index comes first;
 *   weights (tokens x choices floats): scale * s of each, divided by the sum
 *     of the chosen experts' s if renorm (zero where that sum is zero).
 * Scores, choice values and sums are FP64, so that neighbours of a border are
 * told apart as the formula tells them; weights are rounded once to FP32.
 * A choice value of NaN ranks as minus infinity; a logit of minus infinity
 * gives score 0 (a softmax row of nothing else gives NaN weights).
 * SGEMM_MI355_ERR_ROUTE: experts over SGEMM_MI355_MAX_EXPERTS, choices over
 * SGEMM_MI355_MAX_CHOICES or more than stay eligible, groups that do not
 * divide the experts, top_groups outside 1 .. groups. SGEMM_MI355_ERR_OP: an
 * unknown score.
 */
int sgemm_mi355_route(int type, int tokens, int experts, const void *logits, int ld, const float *bias,
                      int score, int groups, int top_groups, int choices, int renorm, float scale,
                      float *weights, int *ids, hipStream_t stream);

/*
 * The gradient of the logits (tokens x experts floats, row stride ldd) for
 * given gradients of the weights (tokens x choices floats). With S the sum of
 * the chosen scores (1 without renorm),
 *   ds_j = scale * (dw_j - renorm * sum_m dw_m s_m / S) / S  on the chosen experts, 0 elsewhere;
 *   softmax: dl_i = s_i * (ds_i - sum_m ds_m s_m);  sigmoid: dl_i = ds_i * s_i * (1 - s_i).
 * The choice itself has no gradient. ids outside 0 .. experts-1 take no part.
 * A token whose S is zero gets zeros.
 */
int sgemm_mi355_route_backward(int type, int tokens, int experts, const void *logits, int ld,
                               const int *ids, const float *dweights, int score, int choices, int renorm, float scale,
                               float *dlogits, int ldd, hipStream_t stream);

/*
 * The rows sorted by expert. ids: tokens x choices ints; row r of the result
 * is the r-th of the tokens*choices entries in order of expert, entries of one
 * expert in their order in ids:
 *   offsets (experts + 1 ints): expert e has rows offsets[e] .. offsets[e+1]-1;
 *   row_token (tokens*choices ints): the token of each row;
 *   place (tokens x choices ints): the row of each entry.
 * Entries whose id is outside 0 .. experts-1 come last, after
 * offsets[experts], in their order; the experts' products make their rows
 * zero. One to three kernels, whose work grows with the entries. `workspace`:
 * device memory of
 * sgemm_mi355_route_plan_workspace_size(tokens, choices, experts) bytes, 4-byte
 * aligned (null where that is 0), free again once the work is done.
 */
int sgemm_mi355_route_plan(int tokens, int choices, int experts, const int *ids,
                           int *offsets, int *row_token, int *place,
                           void *workspace, size_t workspace_bytes, hipStream_t stream);
size_t sgemm_mi355_route_plan_workspace_size(int tokens, int choices, int experts);

/*
 * The experts' rows back to their tokens: y[t] = sum_j weights[t][j] *
 * Z[place[t][j]], summed in FP32 in the order of j and rounded once. Z is rows
 * x cols, Y tokens x cols, both of `type`. A place outside 0 .. rows-1 adds
 * nothing.
 */
int sgemm_mi355_route_combine(int type, int tokens, int choices, int rows, int cols, const void *Z, int ldz,
                              const int *place, const float *weights, void *Y, int ldy, hipStream_t stream);

/*
 * Its gradients: dZ[place[t][j]] = weights[t][j] * dY[t] and dweights[t][j] =
 * sum_n dY[t][n] * Z[place[t][j]][n] (FP32; 0 for a place outside the rows). A row that
 * no place names gets zeros (without any place, nothing is written). No row may
 * be named twice (its gradient would be one of the two):
 * sgemm_mi355_route_plan names each of tokens*choices rows once. dZ has Z's
 * type and row stride lddz. One kernel; two where Z has over 16777216 rows.
 */
int sgemm_mi355_route_combine_backward(int type, int tokens, int choices, int rows, int cols,
                                       const void *dY, int lddy, const void *Z, int ldz, const int *place,
                                       const float *weights, void *dZ, int lddz, float *dweights, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_MI355_ROUTE_H */
