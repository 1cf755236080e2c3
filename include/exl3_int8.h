/*
 * exl3_int8.h - C ABI of the 8-bit integer operators for MI355X (gfx950): quantise,
 * dequantise, a root-mean-square norm that quantises, and the product with an 8-bit
 * weight.  A third weight format beside the trellis (exl3.h) and MXFP4
 * (exl3_mxfp4.h): 8 bits for weights and activations, one scale for each output and
 * each row.
 *
 * Format:
 *   - A row of n values (n % 16 == 0) is n codes, int8 [rows][n], and one scale,
 *     fp32 [rows]; a code c stands for c times its row's scale.  A weight's rows are
 *     its outputs.
 *   - Quantisation of values v with the largest magnitude A: code 127 v / A, the exact
 *     quotient rounded to the nearest whole number, ties to the even one; scale A / 127,
 *     rounded to fp32.  A row of zeros has codes and scale
 *     0.  A row that holds a NaN or an infinity has codes 0 and a scale of NaN: all of
 *     it dequantises to NaN.
 *
 * Conventions: as in exl3.h and exl3_mxfp4.h (device pointers owned by the caller,
 * 16-byte aligned, scales 4-byte aligned, no allocation, `stream` a hipStream_t of the current device,
 * argument errors returned before any launch, no exception crosses, dtype is
 * exl3_dtype).  Results and the workspace share no byte with the arguments or each
 * other (EXL3_EINVAL where they do; the space between the rows of an x is free).
 */
#ifndef EXL3_INT8_H
#define EXL3_INT8_H

#include "exl3_mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows of codes are whole pieces of this many bytes. */
#define EXL3_INT8_PIECE 16

/*
 * exl3_int8_quantize: rows of values to codes and scales.
 *   x      : dtype [rows][n], row r at x + r * ldx elements; ldx >= n, and ldx
 *            times the element size a multiple of 16 bytes
 *   codes  : int8 [rows][n], overwritten
 *   scales : fp32 [rows], overwritten
 * rows == 0 is a no-op.  EXL3_EINVAL for a null or misaligned pointer, a bad dtype,
 * n < 16 or n % 16 != 0, rows < 0 or a bad ldx; EXL3_EUNSUPPORTED for n > 2^24,
 * rows > 2^40 or more than 2^56 values.
 */
int exl3_int8_quantize(const void* x, int32_t dtype, int64_t rows, int32_t n, int64_t ldx, int8_t* codes,
                       float* scales, void* stream);

/*
 * exl3_int8_dequantize: codes times their row's scale, in fp32, rounded to dtype.
 * out: dtype [rows][n], overwritten.  Errors as above; EXL3_EUNSUPPORTED for about
 * 2^36 values and more too.
 */
int exl3_int8_dequantize(const int8_t* codes, const float* scales, int64_t rows, int32_t n, void* out, int32_t dtype,
                         void* stream);

/*
 * exl3_int8_rms_norm: the root-mean-square norm of x + residual, quantised:
 *     h = x + residual, rounded to dtype       (h = x without a residual)
 *     u = h * weight, rounded to fp32
 *     codes, and A / 127, of u as above; scale = A / (127 sqrt(mean(h^2) + eps))
 * so that codes times scale stand for u / sqrt(mean(h^2) + eps).  The mean is over the
 * n values of a row, in 64 bits.
 *   x            : as in exl3_int8_quantize
 *   residual     : NULL, or dtype [rows][n] with the row stride ldr (as ldx)
 *   weight       : weight_dtype [n]
 *   eps          : finite, >= 0
 *   added        : NULL without a residual; with one dtype [rows][n], h, overwritten
 *   codes, scales: as in exl3_int8_quantize; a row in which an h or a u is a NaN or an
 *                  infinity has codes 0 and a scale of NaN, one with no u but zeros 0 and 0
 * rows == 0 is a no-op.  Errors as exl3_int8_quantize; EXL3_EINVAL also for a residual
 * without added or the reverse.
 */
int exl3_int8_rms_norm(const void* x, int32_t dtype, int64_t rows, int32_t n, int64_t ldx, const void* residual,
                       int64_t ldr, const void* weight, int32_t weight_dtype, double eps, int8_t* codes, float* scales,
                       void* added, void* stream);

/*
 * exl3_int8_workspace_bytes: device scratch that exl3_int8_linear needs for `rows`
 * rows of n_in values in n_groups groups (0: none).  EXL3_EINVAL for rows < 0,
 * n_groups < 1 or a bad n_in.  Host-only.
 */
int64_t exl3_int8_workspace_bytes(int32_t rows, int32_t n_groups, int32_t n_in);

/*
 * exl3_int8_matmul: the product of quantised rows with an 8-bit weight,
 *     y[r][o] = (sum_k X[r][k] * W[g(r)][o][k]) * x_scales[r] * scales[g(r)][o],
 * the sum in whole numbers (exact), then converted to fp32, multiplied in this order
 * and rounded to dtype.
 *   x_codes, x_scales : the rows, as exl3_int8_quantize or exl3_int8_rms_norm wrote them
 *   offsets           : NULL (one weight for every row; n_groups == 1), or
 *                       int32 [n_groups + 1], device: rows offsets[g] ..
 *                       offsets[g + 1] - 1 use weight g.  offsets[0] == 0 and
 *                       they do not decrease; rows from offsets[n_groups] on
 *                       belong to no group and come out as zeros.  Values
 *                       outside 0 .. rows are taken as the nearer end.
 *   codes, scales     : the weights, [n_groups][n_out][n_in] and [n_groups][n_out]
 *   y                 : dtype [rows][n_out], overwritten
 * rows == 0 is a no-op.  EXL3_EINVAL for a null or misaligned pointer, a bad dtype,
 * n_in < 16 or n_in % 16 != 0, n_out < 1, rows < 0, n_groups < 1, more than one group
 * without offsets; EXL3_EUNSUPPORTED for n_in >= 2^17 (a sum might pass 32 bits),
 * n_groups > 4096, rows > 2^23, n_out > 2^24, or about 2^36 outputs and more.
 */
int exl3_int8_matmul(const int8_t* x_codes, const float* x_scales, int32_t rows, const int32_t* offsets,
                     int32_t n_groups, const int8_t* codes, const float* scales, int32_t n_in, int32_t n_out, void* y,
                     int32_t dtype, void* stream);

/*
 * exl3_int8_linear: the same product for rows of dtype values, quantised on the way:
 * y equals exl3_int8_matmul of exl3_int8_quantize(x), bit for bit.
 *   x         : dtype [rows][n_in], row stride ldx as in exl3_int8_quantize
 *   workspace : device scratch of exl3_int8_workspace_bytes(rows, n_groups, n_in)
 *               bytes (NULL where that is 0); its contents need no initialisation
 *               and are meaningless after the call.  Calls that may run at the same
 *               time need separate ones.
 * Errors as exl3_int8_matmul, and EXL3_EWORKSPACE.
 */
int exl3_int8_linear(const void* x, int32_t dtype, int32_t rows, int64_t ldx, const int32_t* offsets, int32_t n_groups,
                     const int8_t* codes, const float* scales, int32_t n_in, int32_t n_out, void* y, void* workspace,
                     size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EXL3_INT8_H */
