// Product of microscaled 4-bit weights with 4- or 8-bit activations
// (include/sq_mx.h):
//   y[m, n] = sum_b 2^(ex[m, b] - 127) 2^(ew[n, b] - 127) sum_{k in b} xv wv
// on the matrix cores' scaled f8f6f4 instructions, which multiply a lane's 32
// elements of each operand by that lane's scale byte.
//
// Operand layout (G = 4 lane groups of 16 for 16x16x128, G = 2 of 32 for
// 32x32x64; lane (r, g) serves row r):
//   e2m1  k = 32 g .. 32 g + 31, one 16-byte chunk, low nibble first
//   e4m3  k = 16 g .. + 15 and 16 (G + g) .. + 15, two 16-byte chunks
//   scale of lane (r, g): block g of row r (k = 32 g .. 32 g + 31), both formats
// Weight rows are the instruction's first operand (rows of its result).
#include "mx_device.h"
#include "sq_launch.h"

namespace sq {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int int8x __attribute__((ext_vector_type(8)));

struct MxArgs {
    const uint8_t *xq, *xs, *wq, *ws;
    int M, N, K;
    void *y;
};

template <int YDT>
__device__ __forceinline__ void mx_store_y(void *y, int64_t i, float v) {
    reinterpret_cast<typename OutT<YDT>::T *>(y)[i] = narrow<YDT>(v);
}

__device__ __forceinline__ int8x lo128(int4v a) {  // an e2m1 operand: the upper half is not read
    return __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
}

// One wave per 16 weight rows x 16 tokens, operands straight from memory.
template <int XF, int YDT>
__global__ __launch_bounds__(64) void mx_gemm_plain(MxArgs p) {
    const int lane = threadIdx.x, r = lane & 15, g = lane >> 4;
    const int tn = (p.N + 15) / 16;
    const int n0 = (blockIdx.x % tn) * 16, m0 = (blockIdx.x / tn) * 16;
    const int KB = p.K / 32;
    const int64_t n = n0 + r < p.N ? n0 + r : p.N - 1;
    const int64_t m = m0 + r < p.M ? m0 + r : p.M - 1;
    const int4v *w = reinterpret_cast<const int4v *>(p.wq) + n * KB;
    const uint8_t *ws = p.ws + n * KB, *xs = p.xs + m * KB;
    const int4v *x = reinterpret_cast<const int4v *>(p.xq) + m * KB * (XF == E4M3 ? 2 : 1);
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int b = 0; b < KB; b += 4) {
        const int4v zero = {0, 0, 0, 0};
        const bool in = b + g < KB;
        const int4v wv = in ? w[b + g] : zero;
        const int sw = in ? ws[b + g] : 127, sx = in ? xs[b + g] : 127;
        if constexpr (XF == E2M1) {
            const int4v xv = in ? x[b + g] : zero;
            acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(lo128(wv), lo128(xv), acc, 4, 4,
                                                                    0, sw, 0, sx);
        } else {
            const int c0 = 2 * b + g, c1 = 2 * b + 4 + g;
            const int4v x0 = c0 < 2 * KB ? x[c0] : zero, x1 = c1 < 2 * KB ? x[c1] : zero;
            acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                lo128(wv), __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7), acc, 4, 0, 0,
                sw, 0, sx);
        }
    }
    const int mo = m0 + r;
    if (mo >= p.M) return;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        const int no = n0 + 4 * g + v;
        if (no < p.N) mx_store_y<YDT>(p.y, (int64_t)mo * p.N + no, acc[v]);
    }
}

template <int XF>
static void launch_plain(const MxArgs &a, int y_dt, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)((a.N + 15) / 16) * ((a.M + 15) / 16)));
    if (y_dt == F32) mx_gemm_plain<XF, F32><<<grid, 64, 0, stream>>>(a);
    else if (y_dt == F16) mx_gemm_plain<XF, F16><<<grid, 64, 0, stream>>>(a);
    else mx_gemm_plain<XF, BF16><<<grid, 64, 0, stream>>>(a);
}

void launch_gemm_mx(const uint8_t *xq, const uint8_t *xs, int x_fmt, const uint8_t *wq,
                    const uint8_t *ws, int64_t M, int64_t N, int64_t K, void *y, int y_dt,
                    hipStream_t stream) {
    MxArgs a{};
    a.xq = xq; a.xs = xs; a.wq = wq; a.ws = ws;
    a.M = (int)M; a.N = (int)N; a.K = (int)K; a.y = y;
    if (x_fmt == E2M1) launch_plain<E2M1>(a, y_dt, stream);
    else launch_plain<E4M3>(a, y_dt, stream);
}

}  // namespace sq
