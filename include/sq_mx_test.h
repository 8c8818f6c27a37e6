/*
 * sq_mx_test.h - coverage entry point of the microscaled product: the same
 * call as sq_gemm_mxfp4 (sq_mx.h) with the block shape of its pipelined kernel
 * forced, so that every variant is checked on small shapes.
 */
#ifndef SQ_MX_TEST_H
#define SQ_MX_TEST_H

#include "sq_mx.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * tile -1: the library's choice.  Otherwise, where M > 32 and K >= 256
 * (elsewhere ignored), output tiles of tokens x weight rows:
 *   x_fmt e2m1: 0 256 x 256, 1 256 x 128, 2 128 x 128, 3 64 x 128
 *   x_fmt e4m3: 0 128 x 256, 1 and 2 128 x 128, 3 64 x 128
 * with K % 128 != 0 0 and 1 are 2.  Other values return SQ_ERR_ARG.
 */
int sq_gemm_mxfp4_tile(const uint8_t *xq, const uint8_t *x_scale, int x_fmt, const uint8_t *wq,
                       const uint8_t *w_scale, int64_t M, int64_t N, int64_t K, void *y, int y_dt,
                       void *stream, int tile);

#ifdef __cplusplus
}
#endif

#endif /* SQ_MX_TEST_H */
