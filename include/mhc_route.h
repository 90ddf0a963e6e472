/*
 * mhc_route.h -- C ABI of the routing of tokens to experts on sm_103a: which
 * experts a token takes and with what weight, the gradient of the weights, and
 * the order in which the experts' products take the tokens.
 *
 * Scores.  l: logits [T, E].  s = softmax over the row, or sigmoid of each.  A
 * logit of -inf takes its expert out, as does a bias of -inf; a row of -inf alone
 * (a padded token) takes none.
 *
 * Choice.  key = s, or s + bias (bias [E] steers the choice alone, not the
 * weights).  Without a bias the order is that of the logits.  With groups > 1 the
 * experts are cut into so many runs of E / groups; a group counts for its largest
 * key or for the sum of its two largest (a lone key for itself), and the top_groups
 * best remain.  Of the experts that remain the k with the largest keys are taken,
 * largest first.  Equal keys (-0 and +0 are): the lower index first, for groups too.
 * The order is that of the exact keys of the given fp32 or 16-bit numbers: keys that
 * fp32 cannot tell apart are formed again in fp64.  A NaN counts as larger than any
 * number, so that it is chosen and seen.  Fewer than k experts left: the slots behind
 * hold expert -1 and weight 0.
 *
 * Weights.  w = s of the chosen, divided by their sum if renormalise (formed from
 * ratios, so scores that underflow fp32 still have their shares), times scale;
 * fp32.
 *
 * Backward.  With d = gradient of w and u the unscaled weights:
 *   renormalise    gl_j = scale u_j (d_j - sum_i d_i u_i) h_j on the chosen, else 0;
 *                  h = 1 for softmax, 1 - s_j for sigmoid
 *   softmax        gl_e = scale s_e ([d_e if chosen] - sum_i d_i s_i)
 *   sigmoid        gl_j = scale d_j s_j (1 - s_j) on the chosen, else 0
 * The choice itself has no gradient.  Slots with an expert outside [0, E) count
 * for nothing; one given twice counts twice.
 *
 * Plan.  The slots (t, j) sorted by expert, in slot order within one, each
 * expert's run starting at a multiple of 16 rows: what mhc_experts.h reads.  A slot
 * whose expert is outside [0, E) has no row.
 *
 * Sizes: 0 <= T <= 2^20, T k <= 2^22, E in [1, 1024], 1 <= k <= min(E, 32), groups
 * in [1, 32] and a divisor of E, 1 <= top_groups <= groups, k <= top_groups E /
 * groups.  Tensors are contiguous device memory owned by the caller, aligned to
 * their element; the plan to 256 bytes; the logits of mhc_route_run and grad_logits to
 * four elements where E is a multiple of four and to two where it is even (else
 * MHC_ERR_PARAM_INVALID).  Outputs overlap neither inputs nor one another.  Calls
 * are asynchronous on `stream` (a cudaStream_t, NULL = legacy default) and
 * wait for nothing on the device.  Status codes are those of mhc_pre.h.
 */
#ifndef MHC_ROUTE_H_
#define MHC_ROUTE_H_

#include "mhc_pre.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MHC_DTYPE_FP32 2

#define MHC_SCORE_SOFTMAX 0
#define MHC_SCORE_SIGMOID 1
#define MHC_GROUP_MAX 0
#define MHC_GROUP_TOP2 1

typedef struct {
  int64_t T, E, k;
  int32_t dtype;             /* of logits: MHC_DTYPE_BF16, _FP16 or _FP32     */
  int32_t score;             /* MHC_SCORE_SOFTMAX or MHC_SCORE_SIGMOID        */
  int32_t groups, top_groups;
  int32_t group_score;       /* MHC_GROUP_MAX or MHC_GROUP_TOP2               */
  int32_t renormalise;       /* 0 or 1                                        */
  float scale;
  const void *logits;        /* [T, E]                                        */
  const float *bias;         /* [E] or NULL                                   */
  int32_t *experts;          /* [T, k], written                               */
  float *weights;            /* [T, k], written                               */
} mhc_route_args;

/* Enqueue the routing: one kernel.  T == 0 returns MHC_OK, nothing launched. */
MHC_API mhc_status_t mhc_route_run(const mhc_route_args *a, void *stream);

typedef struct {
  int64_t T, E, k;
  int32_t dtype, score, renormalise;
  float scale;
  const void *logits;          /* [T, E]                                      */
  const int32_t *experts;      /* [T, k]                                      */
  const float *grad_weights;   /* [T, k]                                      */
  void *grad_logits;           /* [T, E], written, the logits' type           */
} mhc_route_bwd_args;

MHC_API mhc_status_t mhc_route_backward_run(const mhc_route_bwd_args *a, void *stream);

/* Device bytes of a plan. */
MHC_API mhc_status_t mhc_expert_plan_size(int64_t T, int64_t k, int64_t E, size_t *bytes);

/* Rows that a plan has room for: T k and up to 15 more for each expert that can
 * have any. */
MHC_API mhc_status_t mhc_expert_plan_rows(int64_t T, int64_t k, int64_t E, int64_t *rows);

/* Enqueue the plan of experts [T, k] into `plan`: one kernel, or three for many
 * slots.  Its words from the 64th on hold the number of slots of each expert
 * (int32 [E]).  T == 0 clears it (experts may be NULL). */
MHC_API mhc_status_t mhc_expert_plan_run(int64_t T, int64_t k, int64_t E, const int32_t *experts, void *plan,
                                         size_t plan_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MHC_ROUTE_H_ */
