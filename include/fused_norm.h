/*
 * fused_norm.h -- C ABI of layer norm (gfx950)
 *
 * The norm in front of a fused linear layer or a router, over the rows of a
 * (M,H) matrix, and its backward pass:
 *
 *   mean = sum_h x / H          rstd = 1 / sqrt(sum_h (x - mean)^2 / H + eps)
 *   xhat = (x - mean) * rstd    y = xhat * weight + bias
 *   g = dy * weight             dx = rstd * (g - sum_h g / H - xhat * sum_h (g * xhat) / H) + R
 *   dweight = sum_rows dy * xhat          dbias = sum_rows dy
 *
 * Conventions are those of fused_linear.h (row-major contiguous operands,
 * caller-owned device pointers, work enqueued on `stream`, no
 * synchronisation, no allocation, arguments validated before any HIP call),
 * with these additions:
 *   Precision  statistics and sums in fp32, one rounding to dtype at the
 *              store; the squares are those of x - mean, and a mean far from
 *              zero (above 16 deviations) is taken to its last place, so it costs no
 *              digits beyond those of x - mean itself.
 *   Values     a row that holds an infinity or a NaN gives NaN throughout
 *              that row and touches no other; so does a row of equal values
 *              with eps 0 (0 * infinity).  The squares are summed in fp32: from
 *              deviations of 2^64 / sqrt(H) on (rows of fp32 or bf16; 2^58 for H =
 *              4096) their sum is infinite and rstd 0, so that y is the bias and dx R or
 *              0; deviations below 2^-75 have no squares, and with eps 0 rstd is infinite.
 *              A row whose sum passes 2^128 is NaN throughout.
 *   Alignment  pointers aligned to their elements (workspace: 16 bytes); any H.
 *   Errors     fl_status as in fused_linear.h; the message of the last failed
 *              call of this header is read with fl_norm_last_error().
 *   Order      every result is the same to the bit from run to run.
 */
#ifndef FUSED_NORM_H
#define FUSED_NORM_H

#include "fused_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Y = the norm of every row of X.
 *   X       (M,H) in dtype.  weight, bias (H,) in dtype, each or NULL (1, 0).
 *   Y       (M,H) in dtype; may equal X.
 *   mean, rstd  (M,) fp32, each or NULL: what the backward pass reads.
 *   eps     finite, not negative.
 * M == 0 or H == 0 writes nothing.
 */
fl_status fl_layer_norm(const void *X, const void *weight, const void *bias, void *Y, float *mean, float *rstd,
                        int64_t M, int64_t H, float eps, fl_dtype dtype, void *stream);

/*
 * The gradients.
 *   dY, X   (M,H) in dtype.  weight (H,) in dtype or NULL.
 *   mean, rstd  (M,) fp32, as fl_layer_norm gave them for X.
 *   R       (M,H) in dtype or NULL: added to dX before its rounding (the
 *           gradient that passes the norm by, where x also goes on as it is).
 *   dX      (M,H) in dtype; may equal dY, X or R.
 *   dweight, dbias  (H,) fp32, each or NULL; overwritten, zeros where M == 0.
 *   workspace  fl_layer_norm_bwd_workspace_bytes(M, H, dtype) bytes (with neither
 *           dweight nor dbias 8 M where H is above 16384, else none), 16-byte
 *           aligned (may be NULL when that is 0); written and read by this
 *           call's launches only, so calls (and captured graphs) that may run at the
 *           same time need one each.
 */
fl_status fl_layer_norm_bwd(const void *dY, const void *X, const void *weight, const float *mean, const float *rstd,
                            const void *R, void *dX, float *dweight, float *dbias, int64_t M, int64_t H,
                            fl_dtype dtype, void *workspace, size_t workspace_bytes, void *stream);
fl_status fl_layer_norm_bwd_workspace_bytes(int64_t M, int64_t H, fl_dtype dtype, size_t *bytes);

const char *fl_norm_last_error(void); /* thread-local; "" when none */

#ifdef __cplusplus
}
#endif

#endif /* FUSED_NORM_H */
