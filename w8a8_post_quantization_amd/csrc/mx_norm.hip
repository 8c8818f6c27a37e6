// Norm -> microscaled codes in one pass over the row (include/sq_mx.h): the
// SmoothQuant tutorial page, section 融入 LayerNorm, as the int8 form in
// norm.hip, with a block scale for every 32 outputs instead of a row step.
//
// Statistics in double from one pass over the registers, with a pivot p (the
// row's first element): S1 = sum (x - p), S2 = sum (x - p)^2,
//   mu = p + S1 / K, sigma^2 = S2 / K - (S1 / K)^2
// (RMS: p = 0, sigma^2 = S2 / K).  The subtraction loses little: one element
// of K gives (p - mu)^2 <= K sigma^2, so S2 / K <= (K + 1) sigma^2 and the
// relative error of sigma^2 stays near K 2^-52 <= 2^-38, against the fp32
// rounding of rstd that follows.
#include "mx_device.h"
#include "sq_launch.h"

namespace sq {

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, kWave);
    return v;
}

template <int DT>
__device__ __forceinline__ float first_of(const void *x, int64_t i) {
    if constexpr (DT == F32) return reinterpret_cast<const float *>(x)[i];
    else if constexpr (DT == F16) return (float)reinterpret_cast<const _Float16 *>(x)[i];
    else return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(x)[i] << 16);
}

// A block per row; thread t holds column groups t + 256 i, i < ITS.
template <int DT, int FMT, int NORM, bool HAS_BETA, int ITS>
__global__ __launch_bounds__(256) void mx_norm_kernel(const void *__restrict__ x, int64_t K,
                                                      const float *__restrict__ gamma,
                                                      const float *__restrict__ beta, float eps,
                                                      uint8_t *__restrict__ q,
                                                      uint8_t *__restrict__ scale) {
    __shared__ double red[2][4];
    const int64_t row = blockIdx.x;
    const int K8 = (int)(K >> 3);
    const int tid = threadIdx.x;
    Raw8<DT> raw[ITS];
#pragma unroll
    for (int i = 0; i < ITS; ++i) {
        const int c = tid + 256 * i;
        raw[i] = load8<DT, false>(x, row * K8 + (c < K8 ? c : K8 - 4 + (tid & 3)));
    }
    const double pivot = NORM == 0 ? (double)first_of<DT>(x, row * K) : 0.0;
    double s1 = 0.0, s2 = 0.0;
#pragma unroll
    for (int i = 0; i < ITS; ++i) {
        float v[8];
        widen8<DT>(raw[i], v);
        if (tid + 256 * i < K8) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const double d = (double)v[k] - pivot;
                if constexpr (NORM == 0) s1 += d;
                s2 = __builtin_fma(d, d, s2);
            }
        }
    }
    s1 = NORM == 0 ? wave_sum(s1) : 0.0;
    s2 = wave_sum(s2);
    if ((tid & 63) == 0) {
        red[0][tid >> 6] = s1;
        red[1][tid >> 6] = s2;
    }
    __syncthreads();
    s1 = red[0][0] + red[0][1] + red[0][2] + red[0][3];
    s2 = red[1][0] + red[1][1] + red[1][2] + red[1][3];
    const double kd = (double)K;
    const double dm = s1 / kd;
    double var = s2 / kd - dm * dm;
    var = var < 0.0 ? 0.0 : var;  // (rounding of a constant row; a NaN stays)
    const float mu = (float)(pivot + dm);
    const float rstd = (float)(1.0 / sqrt(var + (double)eps));
#pragma unroll
    for (int i = 0; i < ITS; ++i) {
        if (256 * i >= K8) break;
        const int c = tid + 256 * i;
        const bool in = c < K8;
        const int cc = in ? c : K8 - 4 + (tid & 3);
        float v[8], g[8], bt[8];
        widen8<DT>(raw[i], v);
        load_f32x8(gamma + cc * 8, g);
        if constexpr (HAS_BETA) load_f32x8(beta + cc * 8, bt);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if constexpr (NORM == 0) v[k] = v[k] - mu;
            v[k] = v[k] * rstd;
            v[k] = v[k] * g[k];
            if constexpr (HAS_BETA) v[k] = v[k] + bt[k];
        }
        uint32_t e;
        const MxCodes<FMT> cd = mx_encode8<FMT>(v, e);
        if (in) mx_store8<FMT, false>(q, scale, row * K8 + c, cd, e);
    }
}

template <int DT, int FMT, int NORM, bool HAS_BETA>
static void launch_mn(const void *x, int64_t M, int64_t K, const float *gamma, const float *beta,
                      float eps, uint8_t *q, uint8_t *scale, hipStream_t stream) {
    const dim3 grid((unsigned)M);
    if (K <= 2048) mx_norm_kernel<DT, FMT, NORM, HAS_BETA, 1><<<grid, 256, 0, stream>>>(x, K, gamma, beta, eps, q, scale);
    else if (K <= 4096) mx_norm_kernel<DT, FMT, NORM, HAS_BETA, 2><<<grid, 256, 0, stream>>>(x, K, gamma, beta, eps, q, scale);
    else if (K <= 8192) mx_norm_kernel<DT, FMT, NORM, HAS_BETA, 4><<<grid, 256, 0, stream>>>(x, K, gamma, beta, eps, q, scale);
    else mx_norm_kernel<DT, FMT, NORM, HAS_BETA, 8><<<grid, 256, 0, stream>>>(x, K, gamma, beta, eps, q, scale);
}

template <int DT, int FMT>
static void launch_mn_kind(const void *x, int64_t M, int64_t K, int norm, const float *gamma,
                           const float *beta, float eps, uint8_t *q, uint8_t *scale,
                           hipStream_t stream) {
    if (norm == 0) {
        if (beta) launch_mn<DT, FMT, 0, true>(x, M, K, gamma, beta, eps, q, scale, stream);
        else launch_mn<DT, FMT, 0, false>(x, M, K, gamma, beta, eps, q, scale, stream);
    } else {
        if (beta) launch_mn<DT, FMT, 1, true>(x, M, K, gamma, beta, eps, q, scale, stream);
        else launch_mn<DT, FMT, 1, false>(x, M, K, gamma, beta, eps, q, scale, stream);
    }
}

template <int DT>
static void launch_mn_fmt(const void *x, int64_t M, int64_t K, int norm, const float *gamma,
                          const float *beta, float eps, int fmt, uint8_t *q, uint8_t *scale,
                          hipStream_t stream) {
    if (fmt == E2M1) launch_mn_kind<DT, E2M1>(x, M, K, norm, gamma, beta, eps, q, scale, stream);
    else launch_mn_kind<DT, E4M3>(x, M, K, norm, gamma, beta, eps, q, scale, stream);
}

void launch_norm_quant_mx(const void *x, int dt, int64_t M, int64_t K, int norm,
                          const float *gamma, const float *beta, float eps, int fmt, uint8_t *q,
                          uint8_t *scale, hipStream_t stream) {
    if (dt == F32) launch_mn_fmt<F32>(x, M, K, norm, gamma, beta, eps, fmt, q, scale, stream);
    else if (dt == F16) launch_mn_fmt<F16>(x, M, K, norm, gamma, beta, eps, fmt, q, scale, stream);
    else launch_mn_fmt<BF16>(x, M, K, norm, gamma, beta, eps, fmt, q, scale, stream);
}

}  // namespace sq
