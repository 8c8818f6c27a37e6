// Norm -> microscaled codes in one pass over the row (include/sq_mx.h): the
// SmoothQuant tutorial page, section 融入 LayerNorm, as the int8 form in
// norm.hip, with a block scale for every 32 outputs instead of a row step.
//
// Statistics in double: S1 = sum x, S2 = sum x^2 in one pass over the
// registers, mu = S1 / K, sigma^2 = S2 / K - mu^2.  The subtraction keeps
// sigma^2 to a relative 2^-53 (K / (64 NW) + 8) mu^2 / sigma^2, so where
// mu^2 > 2^8 sigma^2 a second pass forms sum (x - mu)^2 instead: either way
// the error is below 2^-39 where a row is spread to 32 elements a thread
// (mx_norm_kernel), 2^-37 where a wave holds up to 8192 (mx_norm_wave_kernel),
// against the fp32 rounding of rstd that follows, 2^-24.
// (The fp64 conversions and sums weigh most in the kernel's issue time; a
// pivot subtracted from every element would need no second pass, but one more
// of them for each element.)
#include <type_traits>

#include "mx_device.h"
#include "resident.h"
#include "sq_launch.h"

namespace sq {

// 1 / sqrt(v) for v > 0: the hardware estimate and two Newton steps, within a
// few units of a double's last place (1.0 / sqrt(v) rounds correctly twice,
// in six times the instructions; the result is rounded to fp32 here).
__device__ __forceinline__ double inv_sqrt(double v) {
    double y = __builtin_amdgcn_rsq(v);
    const double h = 0.5 * v;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const double e = __builtin_fma(-h * y, y, 0.5);  // (1 - v y^2) / 2
        y = __builtin_fma(y, e, y);
    }
    return y;
}

// sum / k, rounded: the product with 1 / k alone may be off by a last place, and
// a row of one value v would then have a mean beside v (v = 1 at 35 lengths up to
// 16384, 1568 and 5152 among them, 1.5 at 60) and a sigma^2 above 0.
__device__ __forceinline__ double row_mean(double sum, double k, double inv_k) {
    const double m = sum * inv_k;
    return __builtin_fma(__builtin_fma(-m, k, sum), inv_k, m);
}

// (Newton's steps make NaN of the ends: a zero row with eps = 0 has an infinity
// as defined, a row with an infinity under the RMS norm 0)
__device__ __forceinline__ float row_rstd(double ve) {
    return ve > 0.0 && ve < __builtin_inf() ? (float)inv_sqrt(ve) : (float)(1.0 / sqrt(ve));
}

// The wave's value of lane 63, in every lane.
__device__ __forceinline__ double of_lane63(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, 63);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
    return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

__device__ __forceinline__ void load_f32x8_planes(const float4 *lo, const float4 *hi, float (&m)[8]) {
    const float4 a = *lo, b = *hi;
    m[0] = a.x; m[1] = a.y; m[2] = a.z; m[3] = a.w;
    m[4] = b.x; m[5] = b.y; m[6] = b.z; m[7] = b.w;
}

// NW waves per row; thread t holds column groups t + 64 NW i, i < ITS, and the
// gamma and beta of its columns for all of the block's rows (row b, b + grid,
// ...), the next row's elements in flight meanwhile.  The waves' sums meet in
// LDS slots that alternate between rows: one barrier a row, none for NW = 1.
template <int DT, int FMT, int NORM, bool HAS_BETA, int NW, int ITS, bool NT>
__global__ __launch_bounds__(64 * NW) void mx_norm_kernel(const void *__restrict__ x, int64_t M,
                                                          int64_t K,
                                                          const float *__restrict__ gamma,
                                                          const float *__restrict__ beta, float eps,
                                                          uint8_t *__restrict__ q,
                                                          uint8_t *__restrict__ scale) {
    constexpr int T = 64 * NW;
    __shared__ double red[2][2][NW];
    const int K8 = (int)(K >> 3);
    const int tid = threadIdx.x, wave = tid >> 6;
    int col[ITS];  // (lanes past the row repeat its last block)
    bool in[ITS];
#pragma unroll
    for (int i = 0; i < ITS; ++i) {
        const int c = tid + T * i;
        in[i] = c < K8;
        col[i] = in[i] ? c : K8 - 4 + (tid & 3);
    }
    int64_t row = blockIdx.x;
    Raw8<DT> raw[ITS];
#pragma unroll
    for (int i = 0; i < ITS; ++i) raw[i] = load8<DT, NT>(x, row * K8 + col[i]);
    float g[ITS][8], bt[HAS_BETA ? ITS : 1][8];
#pragma unroll
    for (int i = 0; i < ITS; ++i) {
        load_f32x8(gamma + col[i] * 8, g[i]);
        if constexpr (HAS_BETA) load_f32x8(beta + col[i] * 8, bt[i]);
    }
    const double inv_k = 1.0 / (double)K;
    // (the waves' totals of s1 and s2, in every lane)
    auto total = [&](double &s1, double &s2, int par) __attribute__((always_inline)) {
        if constexpr (NORM == 0) s1 = wave_sum_to_last(s1);
        s2 = wave_sum_to_last(s2);
        if constexpr (NW == 1) {
            if constexpr (NORM == 0) s1 = of_lane63(s1);
            s2 = of_lane63(s2);
        } else {
            if ((tid & 63) == 63) {
                if constexpr (NORM == 0) red[par][0][wave] = s1;
                red[par][1][wave] = s2;
            }
            __syncthreads();
            s1 = 0.0;
            s2 = 0.0;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                if constexpr (NORM == 0) s1 += red[par][0][w];
                s2 += red[par][1][w];
            }
        }
    };
    int par = 0;
    // One row held in `cur`; the next row's loads go to `nxt` first.
    auto one_row = [&](const Raw8<DT> (&cur)[ITS], Raw8<DT> (&nxt)[ITS]) __attribute__((always_inline)) {
        const int64_t next = row + gridDim.x;
        if (next < M) {
#pragma unroll
            for (int i = 0; i < ITS; ++i) nxt[i] = load8<DT, NT>(x, next * K8 + col[i]);
        }
        float v[ITS][8];
        double s1 = 0.0, s2 = 0.0;
#pragma unroll
        for (int i = 0; i < ITS; ++i) {
            widen8<DT>(cur[i], v[i]);
            if (in[i]) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const double d = (double)v[i][k];
                    if constexpr (NORM == 0) s1 += d;
                    s2 = __builtin_fma(d, d, s2);
                }
            }
        }
        total(s1, s2, par);
        par ^= 1;
        const double mean = NORM == 0 ? row_mean(s1, (double)K, inv_k) : 0.0;
        double var = s2 * inv_k - mean * mean;
        if constexpr (NORM == 0) {
            if (mean * mean > 256.0 * var) {  // (uniform over the row's waves)
                double c1 = 0.0, c2 = 0.0;
#pragma unroll
                for (int i = 0; i < ITS; ++i)
                    if (in[i]) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const double d = (double)v[i][k] - mean;
                            c2 = __builtin_fma(d, d, c2);
                        }
                    }
                total(c1, c2, par);
                par ^= 1;
                var = c2 * inv_k;
            }
        }
        const float mu = (float)mean;
        const float rstd = row_rstd(var + (double)eps);
#pragma unroll
        for (int i = 0; i < ITS; ++i) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float y = v[i][k];
                if constexpr (NORM == 0) y = y - mu;
                y = y * rstd;
                y = y * g[i][k];
                if constexpr (HAS_BETA) y = y + bt[i][k];
                v[i][k] = y;
            }
            uint32_t e;
            const MxCodes<FMT> cd = mx_encode8<FMT>(v[i], e);
            if (in[i]) mx_store8<FMT, NT>(q, scale, row * K8 + col[i], cd, e);
        }
        row = next;
    };
    Raw8<DT> other[ITS];
    for (;;) {
        one_row(raw, other);
        if (row >= M) break;
        one_row(other, raw);
        if (row >= M) break;
    }
}

// Many rows of a 16-bit type with a beta, 4096 < K <= 8192: a wave per row and
// no barrier, gamma and beta in LDS (four floats of a group's first half, then
// of its second, so that successive lanes read successive 16 bytes).  With a
// beta the kernel above holds 64 parameters a thread and two blocks a CU;
// 16384 x 7168 fp16, layer norm to e2m1: 66..74 us here, 77 there (RMS norm 61
// and 66; without a beta 66 and 65, RMS 61 and 57: these stay there).  The row
// is held widened (as loaded, and widened again for the output: 72..77 us), in
// 256 registers a thread at two waves a SIMD; four waves in 128 spill (99 us).
// 12.7 VALU instructions an element fill 63 % of the kernel's cycles, and its
// waves, two a SIMD, wait for memory 27 % of theirs (counters).
template <int DT, int FMT, int NORM, int ITS>
__global__ __launch_bounds__(512) void mx_norm_wave_kernel(const void *__restrict__ x, int64_t M,
                                                           int64_t K,
                                                           const float *__restrict__ gamma,
                                                           const float *__restrict__ beta,
                                                           float eps, uint8_t *__restrict__ q,
                                                           uint8_t *__restrict__ scale) {
    static_assert(DT != F32, "16-bit rows");
    constexpr int KMAX8 = ITS * 64;
    __shared__ float4 sg[2][KMAX8], sb[2][KMAX8];
    const int K8 = (int)(K >> 3);
    const int tid = threadIdx.x, lane = tid & 63;
    for (int i = tid; i < 2 * K8; i += 512) {
        sg[i & 1][i >> 1] = reinterpret_cast<const float4 *>(gamma)[i];
        sb[i & 1][i >> 1] = reinterpret_cast<const float4 *>(beta)[i];
    }
    __syncthreads();
    const double inv_k = 1.0 / (double)K;
    for (int64_t row = (int64_t)blockIdx.x * 8 + (tid >> 6); row < M; row += (int64_t)gridDim.x * 8) {
        Raw8<DT> raw[ITS];
#pragma unroll
        for (int i = 0; i < ITS; ++i) {
            const int c = 64 * i + lane;  // (past the row: its last block again)
            raw[i] = load8<DT, true>(x, row * K8 + (c < K8 ? c : K8 - 4 + (lane & 3)));
        }
        float v[ITS][8];
        double s1 = 0.0, s2 = 0.0;
#pragma unroll
        for (int i = 0; i < ITS; ++i) {
            widen8<DT>(raw[i], v[i]);
            if (64 * i + lane < K8) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const double d = (double)v[i][k];
                    if constexpr (NORM == 0) s1 += d;
                    s2 = __builtin_fma(d, d, s2);
                }
            }
            // (kept: the compiler would widen again for the output)
#pragma unroll
            for (int k = 0; k < 8; ++k) asm volatile("" : "+v"(v[i][k]));
        }
        if constexpr (NORM == 0) s1 = of_lane63(wave_sum_to_last(s1));
        s2 = of_lane63(wave_sum_to_last(s2));
        const double mean = NORM == 0 ? row_mean(s1, (double)K, inv_k) : 0.0;
        double var = s2 * inv_k - mean * mean;
        if constexpr (NORM == 0) {
            if (mean * mean > 256.0 * var) {
                double c2 = 0.0;
#pragma unroll
                for (int i = 0; i < ITS; ++i) {
                    if (64 * i + lane < K8) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const double d = (double)v[i][k] - mean;
                            c2 = __builtin_fma(d, d, c2);
                        }
                    }
                }
                var = of_lane63(wave_sum_to_last(c2)) * inv_k;
            }
        }
        const float mu = (float)mean;
        const float rstd = row_rstd(var + (double)eps);
#pragma unroll
        for (int i = 0; i < ITS; ++i) {
            if (64 * i >= K8) break;
            const int c = 64 * i + lane;
            const bool in = c < K8;
            const int cc = in ? c : K8 - 4 + (lane & 3);
            float g[8], bt[8];
            load_f32x8_planes(&sg[0][cc], &sg[1][cc], g);
            load_f32x8_planes(&sb[0][cc], &sb[1][cc], bt);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float y = v[i][k];
                if constexpr (NORM == 0) y = y - mu;
                y = y * rstd;
                y = y * g[k];
                v[i][k] = y + bt[k];
            }
            uint32_t e;
            const MxCodes<FMT> cd = mx_encode8<FMT>(v[i], e);
            if (in) mx_store8<FMT, true>(q, scale, row * K8 + c, cd, e);
        }
    }
}

// As many blocks as the current GPU holds at once, so that all walk down the
// rows together (a second, partial round of blocks would double the time where
// the last round is short).
template <auto Kernel>
static int64_t resident_blocks(int threads) {
    int gpu = -1;
    if (hipGetDevice(&gpu) != hipSuccess) gpu = -1;
    return once_per_gpu<Kernel>(gpu, [&]() -> int64_t {
        int n = 0, cus = 0;
        if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, Kernel, threads, 0) != hipSuccess || n < 1) n = 1;
        if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, gpu) != hipSuccess || cus < 1)
            cus = 256;
        return (int64_t)n * cus;
    });
}

template <int DT, int FMT, int NORM, bool HAS_BETA, int NW, int ITS, bool NT>
static void launch_mn_nt(const void *x, int64_t M, int64_t K, const float *gamma, const float *beta,
                         float eps, uint8_t *q, uint8_t *scale, hipStream_t stream) {
    constexpr auto kernel = mx_norm_kernel<DT, FMT, NORM, HAS_BETA, NW, ITS, NT>;
    const int64_t resident = resident_blocks<kernel>(64 * NW);
    const dim3 grid((unsigned)(M < resident ? M : resident));
    kernel<<<grid, 64 * NW, 0, stream>>>(x, M, K, gamma, beta, eps, q, scale);
}

template <int DT, int FMT, int NORM, bool HAS_BETA, int NW, int ITS>
static void launch_mn_t(const void *x, int64_t M, int64_t K, const float *gamma, const float *beta,
                        float eps, uint8_t *q, uint8_t *scale, hipStream_t stream) {
    if (M * K * dt_bytes(DT) > kNtLoadBytes)
        launch_mn_nt<DT, FMT, NORM, HAS_BETA, NW, ITS, true>(x, M, K, gamma, beta, eps, q, scale, stream);
    else
        launch_mn_nt<DT, FMT, NORM, HAS_BETA, NW, ITS, false>(x, M, K, gamma, beta, eps, q, scale, stream);
}

template <int DT, int FMT, int NORM, bool HAS_BETA>
static void launch_mn(const void *x, int64_t M, int64_t K, const float *gamma, const float *beta,
                      float eps, uint8_t *q, uint8_t *scale, hipStream_t stream) {
    auto go = [&](auto nw, auto its) {
        launch_mn_t<DT, FMT, NORM, HAS_BETA, decltype(nw)::value, decltype(its)::value>(
            x, M, K, gamma, beta, eps, q, scale, stream);
    };
    using std::integral_constant;
    constexpr integral_constant<int, 1> c1;
    constexpr integral_constant<int, 2> c2;
    constexpr integral_constant<int, 4> c4;
    constexpr integral_constant<int, 8> c8;
    if (M <= 512 && K > 512) {
        // few rows: latency; a row spread over up to eight waves
        if (K <= 2048) go(c4, c1);
        else if (K <= 4096) go(c8, c1);
        else if (K <= 8192) go(c8, c2);
        else go(c8, c4);
    } else if (DT != F32 && HAS_BETA && M >= 4096 && K > 4096 && K <= 8192) {
        // (256 blocks of 8 rows: at least two rows a wave.  us so and in the
        // kernel below, layer norm of fp16 to e2m1: 4097 x 7168 21.3 and 24.3,
        // 5120 28.4 and 28.5, 6145 29.9 and 32.8, 16384 66 and 77; 4097 x 4128
        // 14.8 and 20.0, 6000 x 5120 23.1 and 29.3, 8192 x 8192 41.7 and 43.0;
        // RMS norms the same or up to 3 % slower so at 8192 columns; 1024 x 7168
        // 10.4 and 9.2)
        if constexpr (DT != F32 && HAS_BETA)
            mx_norm_wave_kernel<DT, FMT, NORM, 16>
                <<<256, 512, 0, stream>>>(x, M, K, gamma, beta, eps, q, scale);
    } else {
        // many rows: as few waves a row as hold it in four groups a thread
        if (K <= 512) go(c1, c1);
        else if (K <= 1024) go(c1, c2);
        else if (K <= 2048) go(c1, c4);
        else if (K <= 4096) go(c2, c4);
        else if (K <= 8192) go(c4, c4);
        else go(c8, c4);
    }
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
