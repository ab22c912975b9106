/*
 * dobb_layers.h -- C ABI of libdobb.so, continued: the operators of the layers whose weights Dobb trains,
 * a layer norm and a linear map behind it with its operands in 8-bit floating point.
 *
 *   layer norm                dobb_layer_norm, dobb_layer_norm_fp8, dobb_layer_norm_backward
 *   FP8 operands              dobb_fp8_quantize, dobb_fp8_dequantize
 *   products of two of them   dobb_fp8_matmul
 *   captures held in FP8      dobb_accumulate_moment_fp8(_grouped)
 *
 * The conventions of dobb.h hold: device pointers owned by the caller, work enqueued on `stream`
 * without synchronizing, arguments validated on the host before anything is enqueued, results bitwise
 * reproducible for fixed inputs, shapes and device, no state kept between calls.  Every call may be
 * captured into a HIP graph; graphs that share a workspace must be ordered by the caller, as calls are.
 * Buffers that a call writes must not overlap each other or any buffer it reads (DOBB_ERR_INVALID_ARG),
 * unless said otherwise.
 */
#ifndef DOBB_LAYERS_H
#define DOBB_LAYERS_H

#include "dobb.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------------------------------
 * Layer norm over the columns of every row t of X (N x n):
 *   mean_t = sum_c x_tc / n,   rstd_t = (sum_c (x_tc - mean_t)^2 / n + eps)^-1/2,
 *   y_tc = (x_tc - mean_t) rstd_t w_c + b_c
 * X, Y, dY, dX: fp32 or bf16, each of its own type, rows of any stride (ld >= n) aligned to their entries
 * only.  weight, bias: fp32 or bf16 [n] (one type), either NULL for ones or zeros.  mean, rstd: fp32 [N].  A row whose sum
 * of entries, or of squares around the mean, passes fp32's largest value has no mean, or an rstd of 0.
 * Statistics and sums over a row are formed in fp32 around the mean, sums over all rows in fp32 over at most
 * 1024 of them and in fp64 across those; results are rounded once to their type.  eps >= 0; with eps = 0 a row of
 * equal entries has an infinite rstd and NaN results.  NaN and infinities stay within their row, and in the
 * backward pass within their row and the columns' sums.  1 <= N, n <= 2^24.
 * -------------------------------------------------------------------------------------------------*/
/* mean, rstd: either may be NULL.  Y may be X itself (in place) with the same type and stride. */
dobb_status dobb_layer_norm(int64_t N, int64_t n, const void *X, dobb_dtype x_dtype, int64_t ldx, const void *weight,
                            const void *bias, dobb_dtype w_dtype, float eps, void *Y, dobb_dtype y_dtype, int64_t ldy,
                            float *mean, float *rstd, dobb_stream_t stream);
/* Gradients for an output gradient dY, with the mean and rstd of the forward pass: with
 * h = (x - mean) rstd and g = dy w,
 *   dx = rstd (g - mean_c(g) - h mean_c(g h)),   dweight_c = sum_t dy_tc h_tc,   dbias_c = sum_t dy_tc
 * dweight, dbias: g_dtype [n], either NULL where it is not wanted.  dX may be dY itself (in place) with the
 * same type and stride. */
size_t dobb_layer_norm_backward_workspace_size(int64_t N, int64_t n); /* 0: bad arguments */
dobb_status dobb_layer_norm_backward(int64_t N, int64_t n, const void *dY, dobb_dtype dy_dtype, int64_t lddy,
                                     const void *X, dobb_dtype x_dtype, int64_t ldx, const float *mean, const float *rstd,
                                     const void *weight, dobb_dtype w_dtype, void *dX, dobb_dtype dx_dtype, int64_t lddx,
                                     void *dweight, void *dbias, dobb_dtype g_dtype, void *ws, size_t ws_bytes,
                                     dobb_stream_t stream);

/* ------------------------------------------------------------------------------------------------
 * FP8 operands (OCP 8-bit floating point: e4m3, largest value 448, or e5m2, 57344).  An operand holds
 * `rows` rows of k entries, k being the axis that a product contracts, in T = ceil(k / 128) tiles:
 *   codes   T x 8 x rows x 16 bytes: entry [t][h][r] holds entries 128 t + 16 h + 0..15 of row r.
 *           16-byte aligned.
 *   scales  T x R bytes, R = rows rounded up to a multiple of 4: entry [t][r] is the exponent + 127 of the
 *           power of two over row r's entries of tile t (bytes past `rows` are zero).  4-byte aligned.
 * Quantising: 2^e is the least power of two, at least 2^-127, that brings the largest magnitude of its
 * block to the format's largest value or below; code = x / 2^e rounded to the nearest value, ties to
 * even (nothing saturates).  A block is 128 entries along k, or with `square` the 128 x 128 entries of
 * a tile, so that the operands along both axes hold the same values.  A block with a NaN or an infinity gets the
 * scale byte 255 and codes 0x7f (all 128 x 128 with `square`).  The scale byte 255 is NaN, whatever the codes.  Entries past k of other blocks are zeros.  Operands of several micro-batches
 * along their tokens (k) are joined by laying their tiles one behind the other.
 * -------------------------------------------------------------------------------------------------*/
typedef enum { DOBB_E4M3 = 0, DOBB_E5M2 = 1 } dobb_fp8_format;

typedef struct {
    void *codes;
    void *scales;
    int64_t rows, k;             /* 1 <= rows <= 2^24, 1 <= k <= 2^40 */
    dobb_fp8_format format;
} dobb_fp8_operand;

/* X: N x n (ldx >= n), fp32 or bf16, aligned to its entries only; n <= 2^24.  along_rows: the operand of rows N,
 * k = n; along_cols: that of rows n, k = N (a linear layer's input as the operand of its weight's gradient,
 * and as a capture).  Either may be NULL; both hold one format. */
dobb_status dobb_fp8_quantize(int64_t N, int64_t n, const void *X, dobb_dtype x_dtype, int64_t ldx, int32_t square,
                              const dobb_fp8_operand *along_rows, const dobb_fp8_operand *along_cols,
                              dobb_stream_t stream);
/* out: rows x k, or k x rows with `transpose` (fp32 or bf16): the values, exact in fp32 and, from 2^-126 up, in
 * bf16.  DOBB_ERR_SHAPE from 2^36 entries on (whole tiles counted; 2^37 with `transpose`, and 2^38 for dobb_fp8_quantize):
 * more than a launch holds. */
dobb_status dobb_fp8_dequantize(const dobb_fp8_operand *op, int32_t transpose, void *out, dobb_dtype out_dtype,
                                int64_t ldo, dobb_stream_t stream);
/* dobb_layer_norm with its output as FP8 operands: bit for bit dobb_fp8_quantize of the Y that dobb_layer_norm
 * writes in X's type.  mean, rstd are written. */
dobb_status dobb_layer_norm_fp8(int64_t N, int64_t n, const void *X, dobb_dtype x_dtype, int64_t ldx, const void *weight,
                                const void *bias, dobb_dtype w_dtype, float eps, float *mean, float *rstd,
                                const dobb_fp8_operand *along_rows, const dobb_fp8_operand *along_cols,
                                dobb_stream_t stream);

/* ------------------------------------------------------------------------------------------------
 * out (A->rows x B->rows, ldo >= B->rows, fp32 or bf16) = A B^T (+ bias) (+ out if accumulate)
 * for two FP8 operands of the same k, of either format each.  bias: fp32 or bf16 [B->rows] or NULL.  A linear layer
 * y = x W^T takes the operands of x along its rows and of W along its rows; its input's gradient those of dy along its
 * rows and of W along its columns; its weight's gradient those of dy and of x along their columns.  Products are
 * formed on the matrix cores and summed in fp32; the sum, bias and old entry are added in fp32 and
 * rounded once.  For an out in bf16 the matrix instruction multiplies the codes: it adds its products in groups of
 * eight and cuts each at 2^-13 of the group's largest (1.4e-5 of the result for normal entries, where bf16's rounding
 * is 1.7e-3).  For an out in fp32 they are exact, of entries that bf16 holds (below 2^-126 they count as zero).
 * -------------------------------------------------------------------------------------------------*/
size_t dobb_fp8_matmul_workspace_size(int64_t M, int64_t N, int64_t k); /* 0: bad arguments, or no scratch needed */
dobb_status dobb_fp8_matmul(const dobb_fp8_operand *A, const dobb_fp8_operand *B, const void *bias, dobb_dtype bias_dtype,
                            int32_t accumulate, void *out, dobb_dtype out_dtype, int64_t ldo, void *ws, size_t ws_bytes,
                            dobb_stream_t stream);

/* ------------------------------------------------------------------------------------------------
 * dobb_accumulate_moment from captures held as FP8 operands along the columns (rows = s->n, k tokens):
 *   A_b <- beta * A_b + (1 - beta) * (1/N) * sum_t x_{t,b} x_{t,b}^T   over all ceil(k / 128) tiles.
 * N is the divisor, the tokens the tiles hold (1 <= N <= 128 tiles).  Products are exact (entries below
 * 2^-126 count as zero) and summed in fp32 over at most 4096 tokens at a time, four of those sums in fp32 for nb <= 128, the
 * others in fp64.  A (symmetric) is read when beta > 0 and the result is exactly symmetric.  beta is a float, and 1 - beta
 * is taken from it exactly.  Grouped: all operands hold the same number of tiles; captures may be shared by several matrices.
 * -------------------------------------------------------------------------------------------------*/
size_t dobb_moment_fp8_workspace_size(int count, const dobb_shape *shapes, int64_t tiles); /* 0: bad arguments, or no scratch needed */
dobb_status dobb_accumulate_moment_fp8(const dobb_shape *s, const dobb_fp8_operand *op, int64_t N, float beta, float *A,
                                       void *ws, size_t ws_bytes, dobb_stream_t stream);
dobb_status dobb_accumulate_moment_fp8_grouped(int count, const dobb_shape *shapes, const dobb_fp8_operand *ops, int64_t N,
                                               float beta, float *const *A, void *ws, size_t ws_bytes,
                                               dobb_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* DOBB_LAYERS_H */
