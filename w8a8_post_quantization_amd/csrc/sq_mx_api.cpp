// C ABI of the microscaled operators (include/sq_mx.h): argument validation
// on the host, then kernel launches on the caller's stream.
#include "../../include/sq_mx.h"
#include "../../include/sq_mx_test.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "sq_launch.h"

namespace {

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline size_t esize(int dt) { return dt == SQ_F32 ? 4 : 2; }
inline bool valid_dt(int dt) { return dt == SQ_F32 || dt == SQ_F16 || dt == SQ_BF16; }
inline bool valid_fmt(int fmt) { return fmt == SQ_MX_E2M1 || fmt == SQ_MX_E4M3; }
inline hipStream_t st(void *s) { return reinterpret_cast<hipStream_t>(s); }
constexpr int64_t kMaxDim = 0x7fffffff;

inline bool bad_rows(int64_t rows, int64_t K) {
    return rows < 0 || K < 0 || rows > kMaxDim || K > kMaxDim || K % 32 != 0;
}

int finish() { return hipGetLastError() == hipSuccess ? SQ_OK : SQ_ERR_HIP; }

}  // namespace

extern "C" {

int sq_quantize_act_mx(const void *x, int dt, int64_t M, int64_t K, const float *inv_s, int fmt,
                       uint8_t *xq, uint8_t *x_scale, void *stream) {
    if (!valid_dt(dt)) return SQ_ERR_DTYPE;
    if (!valid_fmt(fmt)) return SQ_ERR_ARG;
    if (bad_rows(M, K)) return SQ_ERR_SHAPE;
    if (M == 0) return SQ_OK;
    if (K == 0) return SQ_ERR_SHAPE;  // rows of no elements are rejected
    if (!x || !xq || !x_scale) return SQ_ERR_NULL;
    if (!aligned(x, 16) || !aligned(xq, 16) || !aligned(inv_s, 16) || !aligned(x_scale, 4))
        return SQ_ERR_ALIGN;
    sq::launch_quant_mx(x, dt, M, K, inv_s, nullptr, fmt, xq, x_scale, st(stream));
    return finish();
}

int sq_smooth_weights_mxfp4(const void *w, int dt, int64_t N, int64_t K, const float *row_mul,
                            const float *s, uint8_t *wq, uint8_t *w_scale, void *stream) {
    if (!valid_dt(dt)) return SQ_ERR_DTYPE;
    if (bad_rows(N, K)) return SQ_ERR_SHAPE;
    if (N == 0) return SQ_OK;
    if (K == 0) return SQ_ERR_SHAPE;
    if (!w || !wq || !w_scale) return SQ_ERR_NULL;
    if (!aligned(w, 16) || !aligned(wq, 16) || !aligned(s, 16) || !aligned(row_mul, 4) ||
        !aligned(w_scale, 4))
        return SQ_ERR_ALIGN;
    sq::launch_quant_mx(w, dt, N, K, s, row_mul, SQ_MX_E2M1, wq, w_scale, st(stream));
    return finish();
}

int sq_norm_quantize_act_mx(const void *x, int dt, int64_t M, int64_t K, int norm,
                            const float *gamma, const float *beta, float eps, int fmt,
                            uint8_t *xq, uint8_t *x_scale, void *stream) {
    if (!valid_dt(dt)) return SQ_ERR_DTYPE;
    if (norm != SQ_NORM_LAYER && norm != SQ_NORM_RMS) return SQ_ERR_ARG;
    if (!valid_fmt(fmt)) return SQ_ERR_ARG;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return SQ_ERR_ARG;
    if (bad_rows(M, K)) return SQ_ERR_SHAPE;
    if (M > 0 && K == 0) return SQ_ERR_SHAPE;  // the mean of an empty row is undefined
    if (K > 16384) return SQ_ERR_UNSUPPORTED;
    if (M == 0) return SQ_OK;
    if (!x || !xq || !x_scale || !gamma) return SQ_ERR_NULL;
    if (!aligned(x, 16) || !aligned(xq, 16) || !aligned(gamma, 16) || !aligned(beta, 16) ||
        !aligned(x_scale, 4))
        return SQ_ERR_ALIGN;
    sq::launch_norm_quant_mx(x, dt, M, K, norm, gamma, beta, eps, fmt, xq, x_scale, st(stream));
    return finish();
}

int sq_dequantize_mx(const uint8_t *q, const uint8_t *scale, int fmt, int64_t rows, int64_t K,
                     void *y, int y_dt, void *stream) {
    if (!valid_dt(y_dt)) return SQ_ERR_DTYPE;
    if (!valid_fmt(fmt)) return SQ_ERR_ARG;
    if (bad_rows(rows, K)) return SQ_ERR_SHAPE;
    if (rows == 0) return SQ_OK;
    if (K == 0) return SQ_ERR_SHAPE;
    if (!q || !scale || !y) return SQ_ERR_NULL;
    if (!aligned(q, 16) || !aligned(scale, 4) || !aligned(y, 16)) return SQ_ERR_ALIGN;
    sq::launch_dequant_mx(q, scale, fmt, rows, K, y, y_dt, st(stream));
    return finish();
}

int sq_gemm_mxfp4_tile(const uint8_t *xq, const uint8_t *x_scale, int x_fmt, const uint8_t *wq,
                       const uint8_t *w_scale, int64_t M, int64_t N, int64_t K, void *y, int y_dt,
                       void *stream, int tile) {
    if (tile < -1 || tile > 3) return SQ_ERR_ARG;
    if (!valid_dt(y_dt)) return SQ_ERR_DTYPE;
    if (!valid_fmt(x_fmt)) return SQ_ERR_ARG;
    // (rows and outputs of a last tile past the edge are counted in 32 bits)
    if (bad_rows(M, K) || N < 0 || M > kMaxDim - 1023 || N > kMaxDim - 1023) return SQ_ERR_SHAPE;
    if (M == 0 || N == 0) return SQ_OK;
    if (K == 0) return SQ_ERR_SHAPE;  // an empty inner dimension
    if (K > 1 << 20) return SQ_ERR_UNSUPPORTED;  // 32-bit offsets inside a tile of 256 rows
    if (!xq || !x_scale || !wq || !w_scale || !y) return SQ_ERR_NULL;
    if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(x_scale, 4) || !aligned(w_scale, 4) ||
        !aligned(y, esize(y_dt)))
        return SQ_ERR_ALIGN;
    if (!sq::launch_gemm_mx(xq, x_scale, x_fmt, wq, w_scale, M, N, K, y, y_dt, st(stream), tile))
        return SQ_ERR_UNSUPPORTED;
    return finish();
}

int sq_gemm_mxfp4(const uint8_t *xq, const uint8_t *x_scale, int x_fmt, const uint8_t *wq,
                  const uint8_t *w_scale, int64_t M, int64_t N, int64_t K, void *y, int y_dt,
                  void *stream) {
    return sq_gemm_mxfp4_tile(xq, x_scale, x_fmt, wq, w_scale, M, N, K, y, y_dt, stream, -1);
}

}  // extern "C"
