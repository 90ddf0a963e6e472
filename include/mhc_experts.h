/*
 * mhc_experts.h -- C ABI of routed experts on sm_103a: a layer body of E gated
 * feed-forward blocks of which each token takes a few, forward and backward.
 *
 *   y_t = sum_j w_tj ( act(x_t Wg_e^T) (.) (x_t Wu_e^T) ) Wd_e^T,   e = experts_tj
 *
 * x [T, D], w_gate_up [E, 2, F, D], w_down [E, D, F]: 16-bit tensors of one type,
 * bf16 or fp16; weights [T, k] fp32; act as in mhc_ffn.h.  Which rows an expert
 * takes stands in a plan (mhc_expert_plan_run of mhc_route.h) of the same T, k and
 * E.  Slots without an expert add nothing; a token without any gets a row of zeros.
 *
 * The rows are copied together by expert and taken through two grouped products on
 * the tensor cores (fp32 sums), whose tiles follow the plan, so an expert without
 * rows costs nothing and its weights are not read.  a = act(g) (.) u is rounded to
 * the 16-bit type (operand of the second product; in fp16 it has fp16's range), each
 * expert's output row to 16 significant bits with fp32's range (24-bit rows of the
 * last sum: off by 2^-16 of themselves at most), the weighted sum over a token's
 * experts is formed in fp32 and rounded once.
 *
 * Backward, from g and u as the forward kept them in 16 bits (gate_up [rows, 2, F],
 * rows as in the plan, mhc_expert_plan_rows of them):
 *
 *   ga = grad_y_t Wd_e     grad_weights_tj = sum_f a ga    gg = w ga (.) u (.) act'(g)
 *   gu = w ga (.) act(g)   grad_x_t = sum_j gg Wg_e + gu Wu_e
 *   grad_w_gate_up_e = [gg^T x, gu^T x]      grad_w_down_e = grad_y^T (w a)
 *
 * gg, gu and w a are rounded to the 16-bit type, each expert's row of grad_x to 24
 * bits as an output row is, the gradients once from fp32 sums; an expert without
 * rows gets zero gradients.  Every sum's order follows from the sizes, the plan and
 * the device: results are bitwise reproducible.  Sums over more than 32768 rows are
 * formed in parts joined in fp32.
 *
 * Sizes: D and F multiples of 8 in [8, 16384]; T, k and E as in mhc_route.h.  Tensors
 * are contiguous device memory owned by the caller, 16-byte aligned (weights,
 * grad_weights: 4), workspace and plan 256; outputs and workspace overlap neither
 * inputs nor one another (else MHC_ERR_PARAM_INVALID).  Calls are asynchronous on
 * `stream`.  Status codes are those of mhc_pre.h.
 */
#ifndef MHC_EXPERTS_H_
#define MHC_EXPERTS_H_

#include "mhc_ffn.h"
#include "mhc_route.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int64_t T, E, k, D, F;
  int32_t dtype;             /* MHC_DTYPE_BF16 or MHC_DTYPE_FP16              */
  int32_t act;               /* MHC_FFN_SILU or MHC_FFN_GELU                  */
  const void *x;             /* [T, D]                                        */
  const float *weights;      /* [T, k]                                        */
  const void *plan;
  const void *w_gate_up;     /* [E, 2, F, D]                                  */
  const void *w_down;        /* [E, D, F]                                     */
  void *y;                   /* [T, D], written                               */
  void *gate_up;             /* [rows, 2, F], written where the plan has slots,
                                or NULL                                       */
  void *workspace;           /* device scratch, 256-byte aligned              */
  size_t workspace_bytes;
  uint32_t wait_limit_us;    /* as in mhc_ffn_args                            */
  int32_t withhold_copy;
} mhc_experts_args;

MHC_API mhc_status_t mhc_experts_workspace_size(int64_t T, int64_t E, int64_t k, int64_t D, int64_t F, size_t *bytes);

/* Enqueue the forward: four kernels.  T == 0 returns MHC_OK, nothing launched. */
MHC_API mhc_status_t mhc_experts_run(const mhc_experts_args *a, void *stream);

typedef struct {
  int64_t T, E, k, D, F;
  int32_t dtype, act;
  const void *grad_y;        /* [T, D]                                        */
  const void *x;             /* [T, D]                                        */
  const float *weights;      /* [T, k]                                        */
  const void *plan;
  const void *w_gate_up;     /* [E, 2, F, D]                                  */
  const void *w_down;        /* [E, D, F]                                     */
  const void *gate_up;       /* [rows, 2, F]                                  */
  void *grad_x;              /* [T, D], written                               */
  float *grad_weights;       /* [T, k], written; 0 where there is no expert   */
  void *grad_w_gate_up;      /* [E, 2, F, D], written                         */
  void *grad_w_down;         /* [E, D, F], written                            */
  void *workspace;           /* device scratch, 256-byte aligned              */
  size_t workspace_bytes;
  uint32_t wait_limit_us;
  int32_t withhold_copy;
} mhc_experts_bwd_args;

MHC_API mhc_status_t mhc_experts_backward_workspace_size(int64_t T, int64_t E, int64_t k, int64_t D, int64_t F,
                                                         size_t *bytes);

/* Enqueue the backward: five kernels.  T == 0 writes zeros to both weight gradients
 * (the other tensors but them may be NULL). */
MHC_API mhc_status_t mhc_experts_backward_run(const mhc_experts_bwd_args *a, void *stream);

/* As mhc_ffn_status, for the workspace of either call. */
MHC_API mhc_status_t mhc_experts_status(const void *workspace, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MHC_EXPERTS_H_ */
