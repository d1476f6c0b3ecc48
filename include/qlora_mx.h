/*
 * qlora_mx.h - microscaled floats, RMSNorm and microscaled products of the
 * QLoRA library on AMD Instinct MI355X (gfx950).
 *
 * What serves a model whose adapters have been merged (qlora_nf4_merge): the
 * norm in front of a projection writes its output in microscaled 8-bit
 * floats, and the projection, one for all rows or one per expert, multiplies
 * it with a weight in microscaled 4-bit floats on the matrix cores, which
 * take both operands and their scales as they are stored. The norm also has
 * a bf16 output and a backward pass for training around the QLoRA linear
 * layer.
 *
 * The conventions of qlora_nf4.h hold (row-major contiguous device tensors,
 * 16-byte aligned pointers, caller-owned memory, work enqueued on `stream`,
 * status codes, qlora_last_error), except that NaN and Inf are defined here.
 *
 * Microscaled format (OCP Microscaling Formats specification, version 1.0):
 * blocks of 32 consecutive elements of a row share one power of two.
 *   element  4 bits (sign, 2 exponent bits, bias 1, 1 mantissa bit; largest
 *            magnitude 6) or 8 bits (sign, 4 exponent bits, bias 7, 3
 *            mantissa bits; largest magnitude 448; 0x7f and 0xff are NaN)
 *   scale    one byte s for the factor 2^(s - 127); s = 255 makes every
 *            element of the block NaN
 */
#ifndef QLORA_MX_H
#define QLORA_MX_H

#include <stddef.h>
#include <stdint.h>

#include "qlora_nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define QLORA_MX_BLOCK 32      /* elements per scale */
#define QLORA_MX_EXPERTS 1024  /* most experts of one grouped product */

typedef enum { QLORA_MX_FP4 = 0, QLORA_MX_FP8 = 1 } qlora_mx_type;

/*
 * Microscaled matrix of rows x cols elements (cols a multiple of 32, at most
 * 2^22).
 *   codes   row-major. 4 bits: rows * cols / 2 bytes, element 2j of a row in
 *           the low half of its byte j. 8 bits: rows * cols bytes.
 *   scales  one byte per block, rows of qlora_mx_scale_pitch(cols) =
 *           16 ceil(cols / 512) bytes, so that a row's scales start 16-byte
 *           aligned; the bytes behind a row's cols / 32 scales are 0.
 *   type    a qlora_mx_type
 * The struct lives in host memory, its members are device pointers.
 */
typedef struct {
  int64_t rows, cols;
  uint8_t *codes;
  uint8_t *scales;
  int32_t type;
} qlora_mx_matrix;

/* Bytes between the scales of two rows (0 for an invalid cols). Host-only. */
int64_t qlora_mx_scale_pitch(int64_t cols);

/* Bytes of codes and scales (0 for an invalid shape or type). Host-only. */
size_t qlora_mx_storage_bytes(int64_t rows, int64_t cols, int type);

/*
 * Quantize X [rows, cols] (fp32 or bf16, device) into `out` (same rows and
 * cols, buffers allocated by the caller). Per block, with a the largest
 * magnitude: s = max(floor(log2 a) - e, -127) + 127 with e = 2 (4 bits) or
 * 8 (8 bits), the exponent of the element type's largest power of two
 * (s = 0 for a block of zeros); an element is x / 2^(s - 127) rounded to
 * nearest, ties to the even code, magnitudes past the largest saturating. A
 * zero or an element that rounds to zero keeps its sign. A block that holds
 * a NaN or an Inf gets s = 255 (its codes are unspecified). The pad bytes of
 * the scale rows are written as 0. Results are exact: bit for bit this
 * definition.
 */
int qlora_mx_quantize(const void *X, int x_dtype, int64_t rows, int64_t cols, const qlora_mx_matrix *out, void *stream);

/* Dequantize `q` to out [rows, cols] as fp32 or bf16: element * 2^(s - 127),
 * rounded once where the type cannot hold it (only values below the type's
 * normal range), NaN where s = 255. */
int qlora_mx_dequantize(const qlora_mx_matrix *q, void *out, int out_dtype, void *stream);

/*
 * RMSNorm of the rows of h = bf16(X + residual) (h = X without a residual):
 *     rstd = 1 / sqrt(mean(h^2) + eps),   Y = h * rstd * weight
 * computed in fp64 from the stored bf16 h and rounded once.
 *   X         bf16 [rows, cols]
 *   residual  bf16 [rows, cols] or NULL
 *   weight    fp32 or bf16 (w_dtype) [cols]
 *   eps       finite, >= 0
 *   Y         bf16 [rows, cols]; may be X or residual, not H
 *   H         bf16 [rows, cols], h: needed with a residual, NULL without; may
 *             be X or residual (in place)
 *   rstd      fp32 [rows] for the backward, or NULL
 * cols a multiple of 32, at most 32768. A row that holds a NaN or an Inf has
 * NaN (or 0) outputs and leaves the other rows alone. A row of zeros with
 * eps = 0 is NaN.
 */
int qlora_rmsnorm_fwd(const void *X, const void *residual, const void *weight, int w_dtype, int64_t rows,
                      int64_t cols, double eps, void *Y, void *H, float *rstd, void *stream);

/*
 * The same norm with its output in microscaled floats: Y (same rows and cols)
 * is exactly what qlora_mx_quantize would make of the unrounded Y, with no
 * bf16 rounding in between (a Y below fp32's normal range, 2^-126, is rounded to
 * fp32 first, here and in qlora_rmsnorm_fwd). Y's buffers overlap no input.
 */
int qlora_rmsnorm_mx(const void *X, const void *residual, const void *weight, int w_dtype, int64_t rows,
                     int64_t cols, double eps, const qlora_mx_matrix *Y, void *H, void *stream);

/* Workspace bytes of qlora_rmsnorm_bwd: 0 for a few rows (ws may then be NULL)
 * and for an invalid shape. No contents are expected or kept. */
size_t qlora_rmsnorm_bwd_workspace_bytes(int64_t rows, int64_t cols);

/*
 * Backward of qlora_rmsnorm_fwd, from its h (H, or X where there was no
 * residual) and rstd:
 *     u = h * rstd, g = dY * weight
 *     dX = rstd * (g - u * mean(g * u)) + dH,   dW = sum over rows of dY * u
 *   dH    bf16 [rows, cols], the gradient that reaches h directly (through
 *         the residual stream), or NULL
 *   dX    bf16 [rows, cols]: the gradient of X and of residual; may be dY or
 *         dH (in place), not H
 *   dW    fp32 [cols]
 * fp32 arithmetic; dW's rows are summed in a fixed order (deterministic).
 */
int qlora_rmsnorm_bwd(const void *dY, const void *H, const void *weight, int w_dtype, const float *rstd,
                      const void *dH, int64_t rows, int64_t cols, void *dX, float *dW, void *ws,
                      size_t ws_bytes, void *stream);

/*
 * Y = X W^T: X [M, K] in microscaled 8- or 4-bit floats, W [N, K] in
 * microscaled 4-bit floats, Y bf16 [M, N]. Sums are fp32 in a fixed order
 * (deterministic), Y is rounded once. The elements' products enter the sums
 * exactly, with one reservation that is the matrix instruction's: with an
 * 8-bit X it adds eight neighbouring products of a row at a time and cuts them
 * off 13 binades below the largest of the eight (only products 10 or more
 * binades smaller than it lose anything). M and N are any sizes from 1 to 2^24
 * with M N at most 2^37. A NaN block (scale 255) makes the row (X) or column
 * (W) of Y that it enters NaN, and no other.
 */
int qlora_mx_linear(const qlora_mx_matrix *X, const qlora_mx_matrix *W, void *Y, void *stream);

/*
 * The product by expert: X [M, K] holds rows sorted by expert, W [experts *
 * N, K] the experts' weights one below the other, and
 *     Y[i] = X[i] W_e^T  for offsets[e] <= i < offsets[e + 1]
 *   offsets  int32 [experts + 1] (device), ascending; an expert may have no
 *            row. Rows of Y in front of offsets[0] and from offsets[experts]
 *            on are left as they were. Offsets are read on the GPU only: one
 *            below 0 or past M counts as 0 or M, and an expert whose end lies
 *            before its start has no rows.
 *   experts  1 .. QLORA_MX_EXPERTS, a divisor of W->rows (at most 2^28)
 * Types, sums and sizes as in qlora_mx_linear.
 */
int qlora_mx_linear_grouped(const qlora_mx_matrix *X, const qlora_mx_matrix *W, const int32_t *offsets,
                            int32_t experts, void *Y, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_MX_H */
