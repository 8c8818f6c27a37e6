/*
 * sq_mx.h - microscaled (MX) quantizers and products of the library: 4-bit
 * weights, 4- or 8-bit activations, one power-of-two scale for each block of
 * 32 successive input channels.  Same library (libsq.so), conventions and
 * status codes as sq.h: device pointers owned by the caller, work enqueued on
 * `stream`, arguments checked on the host before anything is enqueued, no
 * allocation, no synchronization, capturable in a HIP graph.
 *
 * The format is the OCP Microscaling one.  A row of K elements (K % 32 == 0)
 * is K / 32 blocks.  Block b holds elements 32 b .. 32 b + 31 and one scale
 * byte e (E8M0): 2^(e - 127), e = 255 for NaN.  Element codes:
 *   SQ_MX_E2M1  4 bits (sign, 2 exponent, 1 mantissa): 0, 0.5, 1, 1.5, 2, 3,
 *               4, 6 and their negatives; element 2 i in the low nibble of
 *               byte i of the row, element 2 i + 1 in the high nibble
 *   SQ_MX_E4M3  8 bits (OCP e4m3fn), largest 448, a byte an element
 * Codes are dense row-major [rows, K / 2] or [rows, K] bytes, scales dense
 * row-major [rows, K / 32] bytes.
 *
 * Quantizing a block of fp32 values v:
 *   a = max |v|, p = floor(log2 a) (-127 for a below 2^-126 or 0)
 *   e = max(p + 127 - P, 0), P = 2 (e2m1) or 8 (e4m3)
 *   code = the format's nearest value to v 2^(127 - e), ties to even,
 *          magnitudes beyond the largest value to the largest
 * Every step is exact or rounds once, so codes and scales do not depend on
 * the kernel.  Unlike the int8 and e4m3 forms of sq.h, inputs need not be
 * finite: a block that holds an infinity or NaN gets e = 255 and codes 0,
 * and every value or product formed from it is NaN.
 *
 * Alignment: x, w, xq, wq, q, s, inv_s, gamma, beta and the y of
 * sq_dequantize_mx 16 bytes; scale bytes and row_mul 4 bytes; the y of
 * sq_gemm_mxfp4 its element size.  Inputs and outputs do not overlap.
 */
#ifndef SQ_MX_H
#define SQ_MX_H

#include "sq.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { SQ_MX_E2M1 = 0, SQ_MX_E4M3 = 1 } sq_mxfmt;

/*
 * a4 in MX: v = fl(X * inv_s), quantized in blocks along K.
 *   x        [M, K] of dt (SQ_F32, SQ_F16 or SQ_BF16)
 *   inv_s    [K] fp32 or NULL (no smoothing)
 *   fmt      SQ_MX_E2M1 or SQ_MX_E4M3
 *   xq, x_scale  out
 * K % 32 == 0; K > 0 when M > 0.  M == 0 enqueues nothing.
 */
int sq_quantize_act_mx(const void *x, int dt, int64_t M, int64_t K, const float *inv_s, int fmt,
                       uint8_t *xq, uint8_t *x_scale, void *stream);

/*
 * a3 in MX (e2m1): v = fl(fl(W * row_mul[n]) * s[k]), quantized in blocks
 * along K.
 *   w        [N, K] of dt
 *   row_mul  [N] fp32 (the next layer's inv_s, as sq_smooth_weights_folded)
 *            or NULL
 *   s        [K] fp32 or NULL
 *   wq [N, K / 2], w_scale [N, K / 32]  out
 * K % 32 == 0; K > 0 when N > 0.
 */
int sq_smooth_weights_mxfp4(const void *w, int dt, int64_t N, int64_t K, const float *row_mul,
                            const float *s, uint8_t *wq, uint8_t *w_scale, void *stream);

/*
 * Norm and MX quantization in one pass: sq_norm_quantize_act's norm with the
 * folded parameters (sq_fold_norm), its output quantized in blocks.
 *   x      [M, K] of dt (SQ_F32, SQ_F16 or SQ_BF16)
 *   norm   SQ_NORM_LAYER: mu = mean_j x_j, sigma^2 = mean_j (x_j - mu)^2;
 *          SQ_NORM_RMS:   mu = 0,          sigma^2 = mean_j x_j^2
 *          summed in double; rstd = 1 / sqrt(sigma^2 + eps) in double; then mu
 *          and rstd rounded to fp32.  The order of the sums depends on M and K
 *          (the same call gives the same bits every time): where a double
 *          result lies at a rounding border, less than one row in 2^13, a
 *          row's mu or rstd may differ in its last place with M.
 *   gamma  [K] fp32; beta [K] fp32 or NULL; eps >= 0, finite
 *   per element in fp32: n = fl(fl(x - mu) * rstd), y = fl(n * gamma_j), then
 *          y = fl(y + beta_j) if beta
 *   fmt, xq, x_scale  as sq_quantize_act_mx, of y
 * K % 32 == 0, 32 <= K <= 16384 when M > 0.
 */
int sq_norm_quantize_act_mx(const void *x, int dt, int64_t M, int64_t K, int norm,
                            const float *gamma, const float *beta, float eps, int fmt,
                            uint8_t *xq, uint8_t *x_scale, void *stream);

/*
 * The values of codes and scales: y = value(code) * 2^(e - 127), narrowed to
 * y_dt with round-to-nearest-even (fp32 holds every value the quantizers
 * produce, bf16 all but those of e4m3 blocks with e < 3, which reach below its
 * smallest subnormal 2^-133; e = 255 gives NaN).
 *   q [rows, K / 2] or [rows, K], scale [rows, K / 32], y [rows, K] of y_dt
 * K % 32 == 0; K > 0 when rows > 0.
 */
int sq_dequantize_mx(const uint8_t *q, const uint8_t *scale, int fmt, int64_t rows, int64_t K,
                     void *y, int y_dt, void *stream);

/*
 * a5 in MX: the product of e2m1 weights with e2m1 or e4m3 activations,
 *   y[m, n] = sum over blocks b of 2^(ex[m, b] - 127) 2^(ew[n, b] - 127)
 *             sum over k in b of xv[m, k] wv[n, k],
 * summed in fp32 on the matrix cores (scaled f8f6f4 instructions, two for a
 * step with e4m3 activations: those of |xv| >= 2 and the others) and narrowed
 * to y_dt with round-to-nearest-even.
 *   xq, x_scale  [M, K] codes and scales of x_fmt (sq_quantize_act_mx or
 *                sq_norm_quantize_act_mx)
 *   wq, w_scale  [N, K] e2m1 (sq_smooth_weights_mxfp4)
 *   y            [M, N] of y_dt
 * The same call gives the same bits every time; the order of the sum depends
 * on M, N and K, so a row's bits may depend on M.  The terms of a step (64 or
 * 128 successive elements) are exact where its blocks' scales are equal, and
 * else within 2^-20 of its largest; an instruction adds them to the fp32 sum in
 * up to four pieces, each cut to the sum's last place.
 * K % 32 == 0, 32 <= K <= 1048576 when M, N > 0 (SQ_ERR_UNSUPPORTED above);
 * M, N <= 2^31 - 1024, in fewer tiles than 2^23 (SQ_ERR_UNSUPPORTED; a tile
 * is 64 x 128 outputs at the least; for K < 256 32 x 32, N <= 16 32 x 16, and
 * fewer than 2^25 of them).
 */
int sq_gemm_mxfp4(const uint8_t *xq, const uint8_t *x_scale, int x_fmt, const uint8_t *wq,
                  const uint8_t *w_scale, int64_t M, int64_t N, int64_t K, void *y, int y_dt,
                  void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SQ_MX_H */
