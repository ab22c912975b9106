/*
 * dobb_ops.h -- C ABI of libdobb.so, continued: the operators a training loop runs around the Dobb
 * step of dobb.h.
 *
 *   gradient norm and clipping   dobb_grad_norm_grouped, dobb_clip_grads_grouped,
 *                                dobb_clip_grad_norm_grouped
 *   captures held in 4 bits      dobb_mx4_quantize, dobb_mx4_dequantize,
 *                                dobb_accumulate_moment_mx4(_grouped)
 *
 * The conventions of dobb.h hold: device pointers owned by the caller, work enqueued on `stream`
 * without synchronizing, arguments validated on the host before anything is enqueued, results bitwise
 * reproducible for fixed inputs, shapes and device, no state kept between calls.  Every call may be
 * captured into a HIP graph; graphs that share a workspace must be ordered by the caller, as calls are.
 */
#ifndef DOBB_OPS_H
#define DOBB_OPS_H

#include "dobb.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------------------------------
 * Global gradient norm over many tensors, and clipping.
 *   norms[i] = sqrt(sum_k G_i[k]^2),   total = sqrt(sum_i norms[i]^2)
 *   out_i[k] = G_i[k] * min(1, max_norm / (total + 1e-6))
 * G: host array of `count` device pointers to dense tensors of numel[i] entries (0 allowed, the pointer
 * may then be NULL) in g_dtypes[i] (fp32 or bf16, mixed lists allowed), aligned to their entries only.
 * The same tensor may be listed twice: it counts twice.  Squares and sums are formed in fp64, so no square of
 * a finite gradient overflows or vanishes; norms and total are rounded to fp32, where one above the largest
 * fp32 value is infinite.  NaN and infinities propagate: a NaN makes total and every clipped gradient NaN; an
 * infinite total makes the coefficient 0 (an infinite entry itself then becomes NaN), or 1 where max_norm is
 * infinite too: no limit changes nothing.
 * norms: device fp32 [count] or NULL.  total: device fp32 scalar.
 * Clipping multiplies in fp32 and rounds to out's type once, to nearest even.  out[i] is G[i] itself
 * with the same dtype (in place: a coefficient of 1 then writes nothing) or a buffer of its own in
 * out_dtypes[i] (fp32 or bf16).  Buffers written (norms, total and the workspace among them) must
 * not overlap each other or any other tensor of the list; a call that breaks this (one tensor listed twice
 * in place, say) is DOBB_ERR_INVALID_ARG.
 * max_norm >= 0, infinity allowed.  dobb_clip_grads_grouped takes the total from device memory, so a
 * caller may combine totals over processes in between; dobb_clip_grad_norm_grouped is the two in a row.
 * -------------------------------------------------------------------------------------------------*/
size_t dobb_grad_norm_workspace_size(int count, const int64_t *numel, const dobb_dtype *g_dtypes); /* 0: bad arguments */
dobb_status dobb_grad_norm_grouped(int count, const int64_t *numel, const void *const *G, const dobb_dtype *g_dtypes,
                                   float *norms, float *total, void *ws, size_t ws_bytes, dobb_stream_t stream);
dobb_status dobb_clip_grads_grouped(int count, const int64_t *numel, const void *const *G, const dobb_dtype *g_dtypes,
                                    void *const *out, const dobb_dtype *out_dtypes, const float *total, float max_norm,
                                    dobb_stream_t stream);
dobb_status dobb_clip_grad_norm_grouped(int count, const int64_t *numel, const void *const *G,
                                        const dobb_dtype *g_dtypes, void *const *out, const dobb_dtype *out_dtypes,
                                        float max_norm, float *norms, float *total, void *ws, size_t ws_bytes,
                                        dobb_stream_t stream);

/* ------------------------------------------------------------------------------------------------
 * Captures in MXFP4 (OCP Microscaling Formats: e2m1 elements, one e8m0 scale per 32).  The scale
 * blocks run along the tokens of one column, the axis the second moment contracts.  N tokens are
 * held in T = ceil(N / 128) tiles of four groups of 32 tokens:
 *   codes   T x 4 x n x 16 bytes: entry [t][g][c] holds column c of tokens 128 t + 32 g + 0..31, two a
 *           byte, the even token in the low half (bit 3 sign, bits 2..1 exponent, bit 0 mantissa:
 *           0, 0.5, 1, 1.5, 2, 3, 4, 6).  16-byte aligned.
 *   scales  T x n x 4 bytes: entry [t][c][g] is that group's scale exponent + 127.  4-byte aligned.
 * Quantising: S = max(floor(log2 max|x|) - 2, -127) over the group, code = x / 2^S rounded to the
 * nearest element, ties to even, above 6 to 6.  A group with a NaN or an infinity gets the scale byte
 * 255 and reads back as NaN.  Tokens past N are zeros.  Captures of several micro-batches with the same
 * n are joined by laying their tiles one behind the other.
 * -------------------------------------------------------------------------------------------------*/
/* X: device, N x n (ldx >= n), fp32 or bf16, aligned to its entries only.  Values, codes and scales that
 * overlap are DOBB_ERR_INVALID_ARG, here and in dobb_mx4_dequantize. */
dobb_status dobb_mx4_quantize(int64_t N, int64_t n, const void *X, dobb_dtype x_dtype, int64_t ldx, void *codes,
                              void *scales, dobb_stream_t stream);
/* out: device, N x n (ldo >= n), fp32 or bf16: the first N tokens' values, exact in fp32 and, from 2^-126
 * up, in bf16. */
dobb_status dobb_mx4_dequantize(int64_t N, int64_t n, const void *codes, const void *scales, void *out,
                                dobb_dtype out_dtype, int64_t ldo, dobb_stream_t stream);
/* dobb_accumulate_moment from a capture in MXFP4:
 *   A_b <- beta * A_b + (1 - beta) * (1/N) * sum_t x_{t,b} x_{t,b}^T   over all `tiles` tiles.
 * N is the divisor, the tokens the tiles hold (1 <= N <= 128 tiles); s->n, s->nb as for
 * dobb_accumulate_moment (n <= 2^24).  Products are formed on the matrix cores and summed in fp32 over at
 * most 16384 tokens, those sums in fp64.  A (symmetric) is
 * read when beta > 0 and the result is exactly symmetric.  beta is a float, as in dobb_accumulate_moment, and
 * 1 - beta is taken from it exactly: 0.9 stands for 0.9f, whose 1 - beta is 2.4e-7 relative above 0.1. */
size_t dobb_moment_mx4_workspace_size(int count, const dobb_shape *shapes, int64_t tiles); /* 0: bad arguments, or no scratch needed */
dobb_status dobb_accumulate_moment_mx4(const dobb_shape *s, const void *codes, const void *scales, int64_t tiles,
                                       int64_t N, float beta, float *A, void *ws, size_t ws_bytes,
                                       dobb_stream_t stream);
/* The same for a matrix set; shapes and pointer arrays are host arrays of length count.  Captures may be
 * shared by several matrices; moments or a workspace that overlap each other or a capture are
 * DOBB_ERR_INVALID_ARG. */
dobb_status dobb_accumulate_moment_mx4_grouped(int count, const dobb_shape *shapes, const void *const *codes,
                                               const void *const *scales, int64_t tiles, int64_t N, float beta,
                                               float *const *A, void *ws, size_t ws_bytes, dobb_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* DOBB_OPS_H */
