/*
 * fused_mx4.h -- C ABI of microscaled 4-bit floating point (gfx950): quantising,
 * reading back, and the fused linear layer over operands held so
 *
 *     out = act(A @ B + bias [+ R])
 *
 * the 4-bit neighbour of fl_fused_linear_fp8, with a scale for every 32 values
 * instead of one for a tensor.
 *
 * Format (MXFP4 of the OCP Microscaling specification 1.0): a row of K values
 * is cut into ceil(K/32) blocks of 32 neighbours, the last filled up with
 * zeros.  A value is a 4-bit E2M1 code: bits 0-2 stand for 0, 0.5, 1, 1.5, 2,
 * 3, 4, 6, bit 3 is the sign.  A block has one E8M0 byte s, the scale
 * 2^(s - 127); 255 stands for NaN.
 *   codes   (rows, 16 * ceil(K/32)) bytes: value 2i of a row in the low half
 *           of its byte i, value 2i+1 in the high half.
 *   scales  (rows, ceil(K/32)) bytes.
 *
 * Conventions are those of fused_linear.h (row-major contiguous operands,
 * caller-owned device pointers, work enqueued on `stream`, no
 * synchronisation, no allocation, arguments validated before any HIP call),
 * with these additions:
 *   Alignment  codes: 16 bytes; scales: any; other pointers: their elements
 *              (workspace: 16 bytes).
 *   Sizes      any up to 2^31 - 1; K up to 2^24 - 256 (the linear layer: below 2^22).
 *   Errors     fl_status as in fused_linear.h; the message of the last failed
 *              call of this header is read with fl_mx4_last_error().
 *   Order      every result is the same to the bit from run to run.
 */
#ifndef FUSED_MX4_H
#define FUSED_MX4_H

#include "fused_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Quantises a matrix.  The scale of a block is 2^(floor(log2 of its largest
 * magnitude) - 2), not below 2^-127; every value over the scale is rounded to
 * the nearest E2M1 value, ties to the even code, above 6 to 6.  A block of
 * zeros has scale byte 0.  A block that holds an infinity or a NaN has scale
 * byte 255 and codes 0: all of it reads as NaN.
 *   X   (rows,K) in dtype, or with transposed (1) a (K,rows) matrix whose
 *       columns become the rows: a weight (K,N) as fl_fused_linear takes it
 *       becomes the B of fl_fused_linear_mx4.
 */
fl_status fl_quantize_mx4(const void *X, uint8_t *codes, uint8_t *scales, int64_t rows, int64_t K, int32_t transposed,
                          fl_dtype dtype, void *stream);

/* X (rows,K) in dtype = the values of codes and scales, rounded once (fp16;
 * values below the smallest step of dtype or above its range: as the
 * rounding has it). */
fl_status fl_dequantize_mx4(const uint8_t *codes, const uint8_t *scales, void *X, int64_t rows, int64_t K,
                            fl_dtype dtype, void *stream);

/*
 * The fused linear layer: X = sum_k A[m,k] B[n,k] + bias (+ R), products exact,
 * summed in fp32; then the activation (the gate with Y), one rounding to
 * dtype and one store.
 *   A, A_scales  M rows of codes and their scales; or, with A_scales NULL, A
 *            (M,K) in dtype, which is quantised on its way in, to the bits
 *            that fl_quantize_mx4 gives.
 *   B, B_scales  N rows of codes and their scales (the weight, K along the row).
 *   bias     (N,) in dtype or NULL.  Y (M,N), for FL_ACT_GLU only.  R (M,N) or
 *            NULL: added before the activation.
 *   out      (M,N) in dtype; may equal Y or R.
 *   dtype    FL_F32, FL_F16 or FL_BF16: of bias, Y, R, out, and of A where it
 *            is given as values.
 *   workspace  fl_mx4_workspace_bytes(M, N, K, A as values, dtype) bytes, 16-byte
 *            aligned (may be NULL when that is 0); written and read by this
 *            call's launches only, so calls (and captured graphs) that may run at the
 *            same time need one each.
 * K == 0 gives act(bias + R); M == 0 or N == 0 writes nothing.  K must be below
 * 2^22, and 256 rows of out span less than 2 GiB.
 */
fl_status fl_fused_linear_mx4(const void *A, const uint8_t *A_scales, const uint8_t *B, const uint8_t *B_scales,
                              const void *bias, const void *Y, const void *R, void *out, int64_t M, int64_t N,
                              int64_t K, fl_act act, fl_dtype dtype, void *workspace, size_t workspace_bytes,
                              void *stream);
fl_status fl_mx4_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t values, fl_dtype dtype, size_t *bytes);

/* How such a call runs: what a workgroup of its launch has of the output. */
typedef struct fl_mx4_plan {
    int32_t kernel;        /* 0 the epilogue alone (no K, or nothing to write), 1 B streamed by few rows of A, 2 tiles */
    int32_t rows, columns; /* of the output */
    int32_t waves;
    int32_t quantize;      /* A's values: 0 there are none, 1 by a launch before, 2 by every workgroup */
    int32_t parts;         /* runs of K, whose sums another launch joins; 1: one */
    int64_t first_columns; /* of the output, in tiles as above; behind them by a second launch; 0: all */
    int32_t second_rows, second_columns, second_waves; /* of that launch, or 0 */
    int32_t reserved;
} fl_mx4_plan;
fl_status fl_mx4_linear_plan(int64_t M, int64_t N, int64_t K, int32_t values, fl_dtype dtype, fl_mx4_plan *plan);

const char *fl_mx4_last_error(void); /* thread-local; "" when none */

#ifdef __cplusplus
}
#endif

#endif /* FUSED_MX4_H */
