/*
 * mhc_post_backward.h -- C ABI of the backward of the mHC post-mapping on
 * sm_103a.
 *
 * The post-mapping (mhc_post.h) is out[t][j][d] = post[t][j] x[t][d] +
 * sum_i comb[t][i][j] residual[t][i][d].  With g the gradient of out:
 *
 *   grad_x[t][d]           = sum_j post[t][j] g[t][j][d]
 *   grad_residual[t][i][d] = sum_j comb[t][i][j] g[t][j][d]
 *   grad_post[t][j]        = sum_d g[t][j][d] x[t][d]
 *   grad_comb[t][i][j]     = sum_d residual[t][i][d] g[t][j][d]
 *
 * All sums are fp32; grad_x and grad_residual are rounded once to bf16
 * (RN-even), grad_post and grad_comb are fp32.  Sums run in an order fixed by
 * T, n, D and the device: results are bitwise reproducible.  grad_x goes to
 * the layer's backward, grad_residual to mhc_pre_backward_run as grad_x_post,
 * grad_post and grad_comb as grad_h_post and grad_h_res.
 *
 * The residual streams are read in bf16, or from an 8-bit checkpoint
 * (mhc_ckpt.h) without being restored first.
 */
#ifndef MHC_POST_BACKWARD_H_
#define MHC_POST_BACKWARD_H_

#include "mhc_pre.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device pointers to contiguous tensors owned by the caller; outputs must not
 * overlap the inputs or one another (else MHC_ERR_PARAM_INVALID). */
typedef struct {
  int64_t T;                 /* tokens; 0 => MHC_OK, nothing launched        */
  int64_t n;                 /* streams, 1..8                                */
  int64_t D;                 /* width, a multiple of 8 in [8, 2^20]          */
  const void *grad_out;      /* bf16 [T, n, D], 16-byte aligned              */
  const void *x;             /* bf16 [T, D], 16-byte aligned                 */
  const void *residual;      /* bf16 [T, n, D], 16-byte aligned, or NULL     */
  const void *codes;         /* uint8 [T, n, D], 8-byte aligned, or NULL      */
  const void *scales;        /* uint8 [T, n, ceil(D/128)], or NULL: a bf16
                                checkpoint, both given exactly when residual
                                is NULL                                      */
  const float *post;         /* fp32 [T, n]                                  */
  const float *comb;         /* fp32 [T, n, n]                               */
  void *grad_x;              /* bf16 [T, D], 16-byte aligned, written        */
  void *grad_residual;       /* bf16 [T, n, D], 16-byte aligned, written     */
  float *grad_post;          /* fp32 [T, n], written                         */
  float *grad_comb;          /* fp32 [T, n, n], written                      */
} mhc_post_bwd_args;

/* Validate, then enqueue one kernel on `stream` (a cudaStream_t, NULL =
 * legacy default).  No workspace, no device-side waits.  MHC_ERR_NULLPTR for
 * a missing tensor, MHC_ERR_PARAM_INVALID for a shape, alignment or
 * residual / checkpoint combination, MHC_ERR_RUNTIME if the launch fails. */
MHC_API mhc_status_t mhc_post_backward_run(const mhc_post_bwd_args *a, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MHC_POST_BACKWARD_H_ */
