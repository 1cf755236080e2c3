/*
 * exl3_mxfp4.h - C ABI of the MXFP4 operators for MI355X (gfx950): quantise,
 * dequantise, and the product with an MXFP4 weight.  They stand beside the
 * trellis operators of exl3.h: a second weight format, for layers that need no
 * calibration and for activations.
 *
 * Format (OCP microscaling, element type E2M1, scale type E8M0, blocks of 32):
 *   - A row of n values (n % 32 == 0) is n / 32 blocks.  Block i has one scale
 *     byte b, which stands for 2^(b - 127) (255: the block is NaN), and 32 codes
 *     of four bits: sign, two exponent bits, one mantissa bit, magnitudes
 *     0, 0.5, 1, 1.5, 2, 3, 4, 6.
 *   - codes: uint8 [rows][n / 2], the code of column 2i in the low half of byte
 *     i; scales: uint8 [rows][n / 32].
 *   - Quantisation: b = max(floor(log2(amax)) - 2 + 127, 0), amax the block's
 *     largest magnitude; a code is the value over 2^(b - 127) rounded to the
 *     nearest magnitude, ties to the even code, at most 6, with the value's
 *     sign (a zero's too).  A block of zeros has b = 0.  A block that holds a
 *     NaN or an infinity has b = 255 and codes 0: it dequantises to NaN.
 *
 * Conventions: as in exl3.h (device pointers owned by the caller, 16-byte
 * aligned, no allocation, `stream` a hipStream_t of the current device,
 * argument errors returned before any launch, no exception crosses).  Results and
 * the workspace share no byte with the arguments or each other (EXL3_EINVAL where
 * they do; the space between the rows of an x is free).  Rows r .. of a weight are
 * one too where its scales are still 16-byte aligned: for r a multiple of 16, or any
 * r where n_in % 512 == 0.  Status codes are exl3_status.
 */
#ifndef EXL3_MXFP4_H
#define EXL3_MXFP4_H

#include "exl3.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of the 16- and 32-bit tensors of a call. */
enum exl3_dtype {
    EXL3_F16 = 0,
    EXL3_BF16 = 1,
    EXL3_F32 = 2
};

/* Values in a block of the format. */
#define EXL3_MXFP4_BLOCK 32

/*
 * exl3_mxfp4_quantize: rows of values to codes and scales.
 *   x      : dtype [rows][n], row r at x + r * ldx elements; ldx >= n, and
 *            ldx times the element size a multiple of 16 bytes
 *   codes  : uint8 [rows][n / 2], overwritten
 *   scales : uint8 [rows][n / 32], overwritten
 * rows == 0 is a no-op.  EXL3_EINVAL for a null or misaligned pointer, a bad
 * dtype, n < 32 or n % 32 != 0, rows < 0 or a bad ldx; EXL3_EUNSUPPORTED for
 * more than 2^37 values.
 */
int exl3_mxfp4_quantize(const void* x, int32_t dtype, int64_t rows, int32_t n, int64_t ldx, uint8_t* codes,
                        uint8_t* scales, void* stream);

/*
 * exl3_mxfp4_dequantize: codes and scales to the values they stand for, rounded
 * to dtype.  Exact in fp32 and bf16 for scale bytes up to 252; at 253 and 254
 * magnitudes of 2^128 and more become infinities, and 255 is NaN.  In fp16 exact
 * for what was quantised from fp16.  out: dtype [rows][n], overwritten.  Errors as
 * above.
 */
int exl3_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t n, void* out,
                          int32_t dtype, void* stream);

/*
 * exl3_mxfp4_workspace_bytes: device scratch that exl3_mxfp4_linear needs for
 * `rows` rows of n_in values in n_groups groups (the quantised rows; 0 where the
 * product quantises them itself).  EXL3_EINVAL for rows < 0, n_groups < 1 or a
 * bad n_in.  Host-only.
 */
int64_t exl3_mxfp4_workspace_bytes(int32_t rows, int32_t n_groups, int32_t n_in);

/*
 * exl3_mxfp4_matmul: the product of quantised rows with an MXFP4 weight,
 *     y[r][o] = sum_k X[r][k] * W[g(r)][o][k],
 * accumulated in fp32 on the matrix cores and rounded once to dtype.
 *   x_codes, x_scales : the rows, as exl3_mxfp4_quantize wrote them
 *   offsets           : NULL (one weight for every row; n_groups == 1), or
 *                       int32 [n_groups + 1], device: rows offsets[g] ..
 *                       offsets[g + 1] - 1 use weight g.  offsets[0] == 0 and
 *                       they do not decrease; rows from offsets[n_groups] on
 *                       belong to no group and come out as zeros.  Values
 *                       outside 0 .. rows are taken as the nearer end.
 *   codes, scales     : the weights, [n_groups][n_out][n_in / 2] and
 *                       [n_groups][n_out][n_in / 32]
 *   y                 : dtype [rows][n_out], overwritten
 * rows == 0 is a no-op.  EXL3_EINVAL for a null or misaligned pointer, a bad
 * dtype, n_in < 32 or n_in % 32 != 0, n_out < 1, rows < 0, n_groups < 1, more
 * than one group without offsets; EXL3_EUNSUPPORTED for n_in > 2^20,
 * n_groups > 4096, rows > 2^23, n_out > 2^24, or about 2^36 outputs and more.
 */
int exl3_mxfp4_matmul(const uint8_t* x_codes, const uint8_t* x_scales, int32_t rows, const int32_t* offsets,
                      int32_t n_groups, const uint8_t* codes, const uint8_t* scales, int32_t n_in, int32_t n_out,
                      void* y, int32_t dtype, void* stream);

/*
 * exl3_mxfp4_linear: the same product for rows of dtype values, quantised on the
 * way: y equals exl3_mxfp4_matmul of exl3_mxfp4_quantize(x), up to fp32
 * summation order.  Few rows are quantised inside the product, one launch;
 * more go through the workspace.
 *   x         : dtype [rows][n_in], row stride ldx as in exl3_mxfp4_quantize
 *   workspace : device scratch of exl3_mxfp4_workspace_bytes(rows, n_groups,
 *               n_in) bytes (NULL where that is 0); its contents need no
 *               initialisation and are meaningless after the call.  Calls that
 *               may run at the same time need separate ones.
 * Errors as exl3_mxfp4_matmul, and EXL3_EWORKSPACE.
 */
int exl3_mxfp4_linear(const void* x, int32_t dtype, int32_t rows, int64_t ldx, const int32_t* offsets,
                      int32_t n_groups, const uint8_t* codes, const uint8_t* scales, int32_t n_in, int32_t n_out,
                      void* y, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EXL3_MXFP4_H */
