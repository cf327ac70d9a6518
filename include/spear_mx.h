/*
 * spear_mx.h - microscaled matrices of libspear, the norm that makes them and
 * the linear layer that multiplies them.
 *
 * Conventions are spear.h's: device pointers owned by the caller, every call
 * asynchronous on the stream it is given, no device memory allocated and
 * nothing copied between host and device, arguments validated on the host
 * before anything is launched, spear_last_error() for the detail.
 */
#ifndef SPEAR_MX_H
#define SPEAR_MX_H

#include "spear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* fp32, where a call of this header or of spear_sample.h allows it beside the
 * two 16-bit types. */
#define SPEAR_F32 2

/*
 * The element formats: 32 consecutive values of a row share a power of two
 * (a byte, exponent + 127) and are held as
 *   SPEAR_MXFP4  e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives,
 *   SPEAR_MXFP8  e4m3: 3 fraction bits, at most 448, steps of 2^-9 below 2^-6
 *                (its codes 0x7F and 0xFF, which quantizing never makes, are NaN).
 * Quantizing takes the power 2^(floor(log2 max|v|) - top), top 2 (fp4) or 8
 * (fp8), not below 2^-127, and rounds v over it to nearest even, saturating.
 * A block of zeros has byte 0.  A block with a value that is not finite has
 * byte 255: all of it reads as NaN, and so do the products that it enters.
 */
typedef enum spear_mx_format { SPEAR_MXFP4 = 0, SPEAR_MXFP8 = 1 } spear_mx_format_t;

/*
 * A microscaled matrix, in the order in which the matrix units take it: rows
 * in blocks of 16, columns in tiles of 128 (4 blocks).  Tile t of row block b
 * is at byte (b * ceil(cols / 128) + t) * 1024 (fp4) or * 2048 (fp8):
 *   fp4  16 (16 i + r) + j / 2: row r, column 32 i + j of the tile, an even j
 *        in the low four bits;
 *   fp8  1024 h + 16 (16 i + r) + j: row r, column 64 h + 16 i + j, j < 16.
 * The scale of row r, columns 32 i .. of tile t is byte
 *   ((b * ceil(cols / 512) + t / 4) * 64 + 16 i + r) * 4 + t % 4.
 * Both arrays are padded to whole tiles, groups of 4 tiles and blocks of rows;
 * padding columns hold zeros with byte 127, padding rows anything.
 *   codes, scales  256-byte aligned, spear_mx_code_bytes and
 *                  spear_mx_scale_bytes long.
 *   rows   0..2^24     cols   1..2^20
 */
typedef struct spear_mx {
  int32_t format; /* a spear_mx_format_t */
  int32_t rows, cols;
  void *codes, *scales;
} spear_mx_t;

/* 0 when the format or a size is invalid (and for rows == 0). */
size_t spear_mx_code_bytes(int32_t format, int32_t rows, int32_t cols);
size_t spear_mx_scale_bytes(int32_t format, int32_t rows, int32_t cols);

/*
 * out = x, quantized: x[r * stride + c] (elements), SPEAR_F16, SPEAR_BF16 or
 * SPEAR_F32, of out's rows and cols; stride >= 0, so rows may repeat.
 */
spear_status_t spear_mx_quantize(const void *x, int32_t dtype, int64_t stride,
                                 const spear_mx_t *out, spear_stream_t stream);

/* out[r * stride + c] = the values of x, rounded once to dtype; stride >= cols
 * where there is more than one row. */
spear_status_t spear_mx_dequantize(const spear_mx_t *x, void *out, int32_t dtype, int64_t stride,
                                   spear_stream_t stream);

/*
 * h = x + residual (fp32; x alone without one), residual_out = h in the type,
 * y = h * r * weight with r = 1 / sqrt(mean(h^2) + eps).  The mean is summed
 * in 64 bits and r rounded once to fp32 (infinite past its range, 2^128, which
 * an eps below 2^-256 allows); the products are fp32, rounded once to the type,
 * or quantized (out_mx).
 *   dtype          SPEAR_F16 or SPEAR_BF16: of x, residual, weight, out.
 *   hidden         1..65536.    rows   0..2^24
 *   strides        between rows, in elements; those of x and residual >= 0.
 *   residual       NULL: none.  residual_out: NULL when residual is; it may be
 *                  residual (or x), the same rows at the same places.
 *   out, out_mx    one of them; out may be x, likewise.
 *   eps            >= 0, finite.
 */
typedef struct spear_norm_args {
  int32_t dtype, rows, hidden;
  const void *x, *residual, *weight;
  int64_t x_stride, residual_stride;
  void *residual_out, *out;
  int64_t residual_out_stride, out_stride;
  const spear_mx_t *out_mx;
  double eps;
} spear_norm_args_t;
spear_status_t spear_rms_norm(const spear_norm_args_t *args, spear_stream_t stream);

/*
 * y[m * y_stride + n] = sum over k of x[m][k] w[n][k], summed in fp32, rounded
 * once to y_dtype (SPEAR_F16, SPEAR_BF16 or SPEAR_F32).  w is SPEAR_MXFP4
 * [N][K]; the tokens are either x_mx [M][K] of either format, or x (16-bit
 * values [M][K], x_stride apart, of x_dtype), which are quantized to x_format
 * first, in the workspace.
 *   y_stride >= N where there is more than one token.
 * One exception to the sum in fp32: 16-bit results of more than 64 SPEAR_MXFP8
 * tokens leave it to the matrix unit's own sum of products of 8 neighbouring
 * columns (8 i .. 8 i + 7), each of which errs by less than 2^-12 of the largest
 * of the eight; about 1.3e-5 of a typical y.  Results in SPEAR_F32 do not.
 */
typedef struct spear_mx_linear_args {
  const spear_mx_t *w;
  const spear_mx_t *x_mx; /* or NULL and: */
  const void *x;
  int32_t x_dtype, x_format, n_tokens;
  int64_t x_stride;
  void *y;
  int32_t y_dtype;
  int64_t y_stride;
} spear_mx_linear_args_t;

/*
 * Workspace bytes that spear_mx_linear needs for this weight and at most
 * n_tokens tokens that come in 16 bits (x_mx needs none: NULL and 0); 0 when
 * an argument is invalid.  256-byte aligned, with any contents; a call on any
 * weight that needs no more may use it.  It overlaps nothing that the call reads
 * or writes; calls that may overlap need different ones.
 */
size_t spear_mx_workspace_bytes(const spear_mx_t *w, int32_t n_tokens);
spear_status_t spear_mx_linear(const spear_mx_linear_args_t *args, void *workspace,
                               size_t workspace_bytes, spear_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEAR_MX_H */
