/*
 * mhc_ckpt.h -- C ABI of the 8-bit activation checkpoints on sm_103a.
 *
 * Hyper-connections keep n residual streams per layer for the backward pass.
 * A checkpoint holds such a 16-bit tensor in 8 bits: each row of D columns is
 * cut into blocks of 128 (the last may be shorter), and a block keeps one
 * exponent e and e4m3 codes of its values:
 *
 *   e     = the smallest integer with amax <= 448 2^e, clamped to the range
 *           of the element type (bf16 [-100, 119], fp16 [-15, 7]); amax is
 *           the largest finite magnitude of the block, and a block without
 *           one (all zero, or nothing finite) takes the range's lower end
 *   code  = e4m3(x 2^-e), ties to even, capped at +-448; an infinity or NaN
 *           becomes the NaN code 0x7F, so that it is still seen when read back
 *   value = code 2^e
 *
 * Inside these ranges every value is exact in the element type, so reading
 * a checkpoint back rounds nothing: the backward pass sees exactly what the
 * 8 bits stand for.  A value is off by at most half a step: 2^-4 of itself, or,
 * where |x| < 2^-6 2^e, 2^-10 2^e.  Magnitudes above 448 times the range's last
 * power (bf16 448 2^119, fp16 57344) become that product: up to an eighth less.
 *
 * codes: uint8 [rows, D].  scales: uint8 [rows, ceil(D / 128)], e + 127.
 *
 * Status codes are those of mhc_pre.h; all tensors are contiguous device
 * memory owned by the caller, outputs apart from inputs and from one another
 * (an overlap gives MHC_ERR_PARAM_INVALID); every call is asynchronous on
 * `stream` (a cudaStream_t, NULL = legacy default stream), needs no workspace
 * and waits for nothing on the device.
 */
#ifndef MHC_CKPT_H_
#define MHC_CKPT_H_

#include "mhc_pre.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MHC_CKPT_BLOCK 128

/* x [rows, D] of dtype (MHC_DTYPE_BF16 or MHC_DTYPE_FP16), 16-byte aligned;
 * D a multiple of 8 in [8, 2^20]; rows >= 0 (0: MHC_OK, nothing launched);
 * codes 8-byte aligned (scales need no alignment).  MHC_ERR_NULLPTR,
 * MHC_ERR_PARAM_INVALID, MHC_ERR_RUNTIME as elsewhere. */
MHC_API mhc_status_t mhc_ckpt8_pack_run(int64_t rows, int64_t D, int32_t dtype, const void *x, void *codes,
                                        void *scales, void *stream);

/* The reverse: x [rows, D] of dtype, written.  A checkpoint is read back in
 * the type it was taken from.  The codes do not hold that type: a bf16 checkpoint
 * read as fp16 is rounded like a cast (out of range: infinite); an fp16 one is
 * exact in bf16 too. */
MHC_API mhc_status_t mhc_ckpt8_restore_run(int64_t rows, int64_t D, int32_t dtype, const void *codes,
                                           const void *scales, void *x, void *stream);

/* mhc_post_run (mhc_post.h) that also writes the checkpoint of its output in
 * the same pass: out is bit for bit that of mhc_post_run, codes [T, n, D] and
 * scales [T, n, ceil(D / 128)] are those of mhc_ckpt8_pack_run on out.  Other
 * arguments and limits as mhc_post_run; codes 8-byte aligned. */
MHC_API mhc_status_t mhc_post_ckpt_run(int64_t T, int64_t n, int64_t D, const void *x, const void *residual,
                                       const float *post, const float *comb, void *out, void *codes, void *scales,
                                       void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MHC_CKPT_H_ */
