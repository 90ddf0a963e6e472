/*
 * mhc_ffn.h -- C ABI of the gated feed-forward block on sm_103a, forward and
 * backward: the layer body between the pre-mapping's y and the post-mapping's
 * x.
 *
 *   g = x Wg^T    u = x Wu^T    a = act(g) (.) u    y = a Wd^T
 *
 * x [T, D], w_gate_up [2, F, D] (Wg, then Wu), w_down [D, F]: 16-bit tensors of
 * one type, bf16 or fp16.  act is silu, z / (1 + e^-z), or gelu in its tanh
 * form, 0.5 z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))).  Both projections, the
 * activation and the product are one kernel; the products run on the tensor
 * cores with fp32 sums; exponential and division are the fast ones, a few 2^-22
 * of their results off.  a is rounded to the 16-bit type (it is an operand of the
 * second product), y once from its fp32 sum: y is off by about 1.4 times what one
 * rounding of exact values would leave.  In fp16, a has fp16's range as well: a
 * product act(g) u above 65504 is infinite, whatever y would be.
 *
 * For the backward pass the forward can keep g and u, rounded to 16 bits
 * (gate_up [T, 2, F]) or in 8 bits (codes [T, 2, F] and scales
 * [T, 2, ceil(F / 128)], the checkpoint form of mhc_ckpt.h taken from the fp32
 * sums).  With g and u what was kept:
 *
 *   ga = grad_y Wd        gg = ga (.) u (.) act'(g)      gu = ga (.) act(g)
 *   grad_x = gg Wg + gu Wu                 grad_w_gate_up = [gg^T x, gu^T x]
 *   grad_w_down = grad_y^T a               a = act(g) (.) u, formed again
 *
 * gg, gu and a are rounded to the 16-bit type (in fp16 also to its range: above
 * 65504 infinite, below 6e-8 zero, so small gradients want a scaled loss), the
 * gradients once from their fp32 sums.  Sums run in an order fixed by the sizes and the device: results
 * are bitwise reproducible.  The tensor cores truncate as they add: sums of terms
 * of one sign measured 1e-7 of the sum too small for every sixteen terms.  Sums over more than 32768 tokens, and sums over F and 2F that are
 * deeper than that, are formed in parts joined in fp32, so that this stays below
 * 2.2e-4; sums over D, and those over F for up to 128 tokens, are not cut so.
 *
 * Sizes: D and F multiples of 8 in [8, 2^20], 0 <= T <= 2^24.  Every tensor is
 * contiguous device memory owned by the caller, 16-byte aligned (scales: no
 * alignment); outputs and workspace overlap neither inputs nor one another (else
 * MHC_ERR_PARAM_INVALID).  Calls are asynchronous on `stream` (a cudaStream_t,
 * NULL = legacy default).  Status codes are those of mhc_pre.h.
 */
#ifndef MHC_FFN_H_
#define MHC_FFN_H_

#include "mhc_pre.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MHC_FFN_SILU 0
#define MHC_FFN_GELU 1

typedef struct {
  int64_t T, D, F;
  int32_t dtype;             /* MHC_DTYPE_BF16 or MHC_DTYPE_FP16              */
  int32_t act;               /* MHC_FFN_SILU or MHC_FFN_GELU                  */
  const void *x;             /* [T, D]                                        */
  const void *w_gate_up;     /* [2, F, D]                                     */
  const void *w_down;        /* [D, F]                                        */
  void *y;                   /* [T, D], written                               */
  void *gate_up;             /* [T, 2, F], written, or NULL                   */
  void *codes;               /* uint8 [T, 2, F], written, or NULL             */
  void *scales;              /* uint8 [T, 2, ceil(F/128)]; with codes only; at
                                most one of gate_up and codes is given        */
  void *workspace;           /* device scratch, 256-byte aligned              */
  size_t workspace_bytes;
  uint32_t wait_limit_us;    /* device wait limit; 0: the default, 2 s; at most 10 s.
                                A bound on hangs: it has to exceed the time that
                                one block takes for its share of one product
                                (hundreds of microseconds for weights of several
                                GB); the time of an earlier product of the call
                                does not count                                */
  int32_t withhold_copy;     /* 1: leave out one operand copy, so that the waits
                                on it give up (test of that path; outputs are
                                then incomplete); 0 otherwise                 */
} mhc_ffn_args;

/* Device scratch of a forward call: a 256-byte header (its first word is the
 * error word), a [T, F] and, where the second product is cut along its depth, fp32
 * sums of the parts.  T == 0 gives 0. */
MHC_API mhc_status_t mhc_ffn_workspace_size(int64_t T, int64_t D, int64_t F, size_t *bytes);

/* Enqueue the forward: two kernels (three where parts are joined).  T == 0 returns MHC_OK, nothing launched.
 * MHC_ERR_NULLPTR for a missing tensor, MHC_ERR_PARAM_INVALID for sizes, types,
 * alignment or workspace, MHC_ERR_RUNTIME for no sm_103 device or a launch
 * failure. */
MHC_API mhc_status_t mhc_ffn_run(const mhc_ffn_args *a, void *stream);

typedef struct {
  int64_t T, D, F;
  int32_t dtype, act;
  const void *grad_y;        /* [T, D]                                        */
  const void *x;             /* [T, D]                                        */
  const void *w_gate_up;     /* [2, F, D]                                     */
  const void *w_down;        /* [D, F]                                        */
  const void *gate_up;       /* [T, 2, F], or NULL                            */
  const void *codes;         /* uint8 [T, 2, F], or NULL                      */
  const void *scales;        /* with codes; exactly one form is given         */
  void *grad_x;              /* [T, D], written                               */
  void *grad_w_gate_up;      /* [2, F, D], written                            */
  void *grad_w_down;         /* [D, F], written                               */
  void *workspace;           /* device scratch, 256-byte aligned              */
  size_t workspace_bytes;
  uint32_t wait_limit_us;    /* as in mhc_ffn_args                            */
  int32_t withhold_copy;
} mhc_ffn_bwd_args;

/* Device scratch of a backward call: the header, [gg, gu] [T, 2, F], a [T, F]
 * and, for each gradient that is cut along its depth, fp32 sums of the parts. */
MHC_API mhc_status_t mhc_ffn_backward_workspace_size(int64_t T, int64_t D, int64_t F, size_t *bytes);

/* Enqueue the backward: two to three kernels, and one more for each gradient whose
 * parts are joined.  T == 0 writes zeros to both weight
 * gradients (x, grad_y, grad_x and the kept sums may be NULL). */
MHC_API mhc_status_t mhc_ffn_backward_run(const mhc_ffn_bwd_args *a, void *stream);

/* Synchronise `stream`, then MHC_ERR_RUNTIME if a CUDA error is pending or the
 * error word of the last call that used `workspace` is set (a device wait that
 * gave up), else MHC_OK.  workspace NULL: only the stream is checked. */
MHC_API mhc_status_t mhc_ffn_status(const void *workspace, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MHC_FFN_H_ */
