/*
 * mhc_orth.h -- C ABI of the orthogonalised update on sm_103a: the matrix of an
 * update (a momentum, a gradient) brought near the closest matrix with orthonormal
 * rows or columns by Newton-Schulz products, as optimisers of matrix weights take it.
 *
 *   X = G / (|G| + eps),   |G|: root of the sum of squares
 *   for each step (a, b, c):   A = X X^T,   X <- a X + (b A + c A A) X
 *
 * (with A = X^T X from the other side where G is taller than wide: the same result).
 * Each step maps every singular value s of X to a s + b s^3 + c s^5.
 *
 * x [batch, rows, cols] fp32, bf16 or fp16; out of the same shape, bf16 or fp16.
 * The norm is summed in fp32 beside powers of two (compensated) and fp64, whatever the
 * magnitudes.  X, A and b A + c A A are held in fp16 between the products (11 bits where
 * bf16 has 8), scaled by powers of two into its range, what the two diagonals lose by it in
 * fp32 beside them; products are summed in fp32, X <- ... is formed in fp32 and rounded
 * once.  A result is off by about 2^-12 of its rows' size for each rounding,
 * more for directions much weaker than the strongest (a singular value r times
 * smaller: r times as much of itself).  Singular values have to stay below 1.6:
 * the coefficients are the caller's to choose so (those in use stay below 1.3).  A zero matrix
 * gives zeros; one with an infinity or NaN gives NaN.  Results are bitwise
 * reproducible; of a matrix in batches of different sizes the sums' order may differ.
 *
 * Sizes: batch in [0, 65535], rows and cols in [1, 32768], 1 to 32 steps.  x and out
 * contiguous device memory aligned to their element; out and workspace overlap neither x
 * nor one another.  Calls are asynchronous on `stream`.  Status codes are those of
 * mhc_pre.h.
 */
#ifndef MHC_ORTH_H_
#define MHC_ORTH_H_

#include "mhc_route.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int64_t batch, rows, cols;
  int32_t dtype;             /* of x: MHC_DTYPE_BF16, _FP16 or _FP32          */
  int32_t out_dtype;         /* MHC_DTYPE_BF16 or MHC_DTYPE_FP16              */
  int32_t steps;
  float eps;                 /* >= 0                                          */
  const float *coefficients; /* host, [steps, 3]: a, b, c of each step        */
  const void *x;             /* [batch, rows, cols]                           */
  void *out;                 /* [batch, rows, cols], written                  */
  void *workspace;           /* device scratch, 256-byte aligned              */
  size_t workspace_bytes;
  uint32_t wait_limit_us;    /* as in mhc_ffn_args                            */
  int32_t withhold_copy;
} mhc_orth_args;

MHC_API mhc_status_t mhc_orth_workspace_size(int64_t batch, int64_t rows, int64_t cols, size_t *bytes);

/* Enqueue: two kernels and three for each step, four where few deep tiles of X X^T are
 * summed in parts.  batch == 0 returns MHC_OK, nothing launched. */
MHC_API mhc_status_t mhc_orth_run(const mhc_orth_args *a, void *stream);

/* As mhc_ffn_status. */
MHC_API mhc_status_t mhc_orth_status(const void *workspace, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MHC_ORTH_H_ */
