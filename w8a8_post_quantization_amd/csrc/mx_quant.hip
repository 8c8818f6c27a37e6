// Microscaled (MX) row quantizer with the smoothing fused into the read, and
// its inverse (include/sq_mx.h):
//   v = fl(fl(x[r, k] * row_mul[r]) * mul[k]);  per block of 32 successive k:
//   a = max |v|, e = max(exponent(a) - P, 0), code = nearest(v 2^(127 - e))
// A block's scale needs nothing from the rest of the row, so unlike the
// per-row quantizers there is no row reduction: a lane takes eight elements
// (one 16-byte load of a 16-bit type), a quad of lanes one block.
#include "mx_device.h"
#include "sq_launch.h"

namespace sq {

// Threads are CW column groups (of eight elements) by 256 / CW rows; a block
// covers CW column groups and walks down its rows, so that each thread's
// multipliers stay in registers.  K % 32 == 0: a quad is all inside the row
// or all outside, and every lane converts (lanes outside on a clamped
// column), since the block maximum reads its quad.
// Bound by memory: 28672 x 7168 fp16 to e2m1 with both multipliers 96 us, 520 MB
// at 5.4 TB/s (a 2 : 1 mix of plain reads and writes reaches 6.15).
template <int DT, int FMT, bool HAS_MUL, bool HAS_ROW, int CW, bool NT>
__global__ __launch_bounds__(256) void mx_quant_kernel(const void *__restrict__ x, int64_t rows,
                                                       int64_t K, const float *__restrict__ mul,
                                                       const float *__restrict__ row_mul,
                                                       uint8_t *__restrict__ q,
                                                       uint8_t *__restrict__ scale, int slabs,
                                                       int64_t rows_per_block) {
    constexpr int RW = 256 / CW;
    const int64_t K8 = K >> 3;
    const int64_t slab = blockIdx.x % slabs;
    const int64_t r0 = (int64_t)(blockIdx.x / slabs) * rows_per_block;
    const int64_t r1 = r0 + rows_per_block < rows ? r0 + rows_per_block : rows;
    int64_t c8 = slab * CW + threadIdx.x % CW;
    const bool in = c8 < K8;
    c8 = in ? c8 : K8 - 4 + (threadIdx.x & 3);
    float m[8];
    if constexpr (HAS_MUL) load_f32x8(mul + c8 * 8, m);
    constexpr int U = 4;  // rows in flight
    for (int64_t rb = r0 + threadIdx.x / CW; rb < r1; rb += RW * U) {
        Raw8<DT> raw[U];
        float rm[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = rb + u * RW < r1 ? rb + u * RW : r1 - 1;
            raw[u] = load8<DT, NT>(x, r * K8 + c8);
            if constexpr (HAS_ROW) rm[u] = row_mul[r];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[8];
            widen8<DT>(raw[u], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if constexpr (HAS_ROW) v[i] = v[i] * rm[u];
                if constexpr (HAS_MUL) v[i] = v[i] * m[i];
            }
            uint32_t e;
            const MxCodes<FMT> c = mx_encode8<FMT>(v, e);
            if (in && rb + u * RW < r1) mx_store8<FMT, NT>(q, scale, (rb + u * RW) * K8 + c8, c, e);
        }
    }
}

template <int DT, int FMT, bool HAS_MUL, bool HAS_ROW, int CW>
static void launch_mq(const void *x, int64_t rows, int64_t K, const float *mul,
                      const float *row_mul, uint8_t *q, uint8_t *scale, hipStream_t stream) {
    constexpr int RW = 256 / CW;
    const int slabs = (int)((K / 8 + CW - 1) / CW);
    // enough blocks to fill the chip several times, and whole groups of rows
    int64_t groups = (8192 + slabs - 1) / slabs;
    int64_t per = (rows + groups - 1) / groups;
    per = (per + RW - 1) / RW * RW;
    groups = (rows + per - 1) / per;
    const dim3 grid((unsigned)(groups * slabs));
    if (rows * K * dt_bytes(DT) > kNtLoadBytes)
        mx_quant_kernel<DT, FMT, HAS_MUL, HAS_ROW, CW, true>
            <<<grid, 256, 0, stream>>>(x, rows, K, mul, row_mul, q, scale, slabs, per);
    else
        mx_quant_kernel<DT, FMT, HAS_MUL, HAS_ROW, CW, false>
            <<<grid, 256, 0, stream>>>(x, rows, K, mul, row_mul, q, scale, slabs, per);
}

template <int DT, int FMT, bool HAS_MUL, bool HAS_ROW>
static void launch_mq_cw(const void *x, int64_t rows, int64_t K, const float *mul,
                         const float *row_mul, uint8_t *q, uint8_t *scale, hipStream_t stream) {
    if (K >= 512) launch_mq<DT, FMT, HAS_MUL, HAS_ROW, 64>(x, rows, K, mul, row_mul, q, scale, stream);
    else launch_mq<DT, FMT, HAS_MUL, HAS_ROW, 4>(x, rows, K, mul, row_mul, q, scale, stream);
}

template <int DT>
static void launch_mq_dt(const void *x, int64_t rows, int64_t K, const float *mul,
                         const float *row_mul, int fmt, uint8_t *q, uint8_t *scale,
                         hipStream_t stream) {
    if (fmt == E4M3) {
        if (mul) launch_mq_cw<DT, E4M3, true, false>(x, rows, K, mul, nullptr, q, scale, stream);
        else launch_mq_cw<DT, E4M3, false, false>(x, rows, K, mul, nullptr, q, scale, stream);
    } else if (row_mul) {
        if (mul) launch_mq_cw<DT, E2M1, true, true>(x, rows, K, mul, row_mul, q, scale, stream);
        else launch_mq_cw<DT, E2M1, false, true>(x, rows, K, mul, row_mul, q, scale, stream);
    } else {
        if (mul) launch_mq_cw<DT, E2M1, true, false>(x, rows, K, mul, nullptr, q, scale, stream);
        else launch_mq_cw<DT, E2M1, false, false>(x, rows, K, mul, nullptr, q, scale, stream);
    }
}

void launch_quant_mx(const void *x, int dt, int64_t rows, int64_t K, const float *mul,
                     const float *row_mul, int fmt, uint8_t *q, uint8_t *scale,
                     hipStream_t stream) {
    if (dt == F32) launch_mq_dt<F32>(x, rows, K, mul, row_mul, fmt, q, scale, stream);
    else if (dt == F16) launch_mq_dt<F16>(x, rows, K, mul, row_mul, fmt, q, scale, stream);
    else launch_mq_dt<BF16>(x, rows, K, mul, row_mul, fmt, q, scale, stream);
}

// ------------------------------------------------------------------ inverse

// y = value(code) 2^(e - 127), exact in fp32, then narrowed.  Rows are dense
// and hold whole blocks, so the arrays are read flat: lane i takes the i-th
// group of E elements, as many as make one 16-byte store (32 bytes of fp32 a
// lane in two stores, each of every other 16 bytes: 95 us against 44 for
// 8192 x 7168 e4m3).  28672 x 7168 e2m1 to fp16 96 us, 5.4 TB/s.
template <int FMT, int E>
__device__ __forceinline__ void mx_decode(const uint32_t *c, uint32_t e, float (&v)[E]) {
    const float s = __uint_as_float(e > 0 ? (e == 255u ? 0x7fc00000u : e << 23) : 0x00400000u);
    typedef float f2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int h = 0; h < E / 4; ++h) {
        f2 lo, hi;
        if constexpr (FMT == E2M1) {  // (the byte of the word is an immediate)
            lo = h == 0 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[0], 1.0f, 0)
                        : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[0], 1.0f, 2);
            hi = h == 0 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[0], 1.0f, 1)
                        : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[0], 1.0f, 3);
        } else {
            lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[h], false);
            hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[h], true);
        }
        v[4 * h] = lo[0] * s;
        v[4 * h + 1] = lo[1] * s;
        v[4 * h + 2] = hi[0] * s;
        v[4 * h + 3] = hi[1] * s;
    }
}

template <int FMT, int YDT, bool NT>
__global__ __launch_bounds__(256) void mx_dequant_kernel(const uint8_t *__restrict__ q,
                                                         const uint8_t *__restrict__ scale,
                                                         int64_t n, void *__restrict__ y) {
    constexpr int U = 4, E = Vec<YDT>::n;  // groups in flight, elements a group
    using T = typename OutT<YDT>::T;
    for (int64_t b = (int64_t)blockIdx.x * (256 * U); b < n; b += (int64_t)gridDim.x * (256 * U)) {
        uint32_t c[U][2], e[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            int64_t i = b + u * 256 + threadIdx.x;
            i = i < n ? i : n - 1;
            if constexpr (FMT == E2M1 && E == 4) {
                c[u][0] = reinterpret_cast<const uint16_t *>(q)[i];
            } else if constexpr (FMT == E4M3 && E == 8) {
                const uint2 t = reinterpret_cast<const uint2 *>(q)[i];
                c[u][0] = t.x;
                c[u][1] = t.y;
            } else {
                c[u][0] = reinterpret_cast<const uint32_t *>(q)[i];
            }
            e[u] = scale[i / (32 / E)];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = b + u * 256 + threadIdx.x;
            if (i >= n) break;
            float v[E];
            mx_decode<FMT, E>(c[u], e[u], v);
            T h[E];
#pragma unroll
            for (int k = 0; k < E; ++k) h[k] = narrow<YDT>(v[k]);
            u4v *p = reinterpret_cast<u4v *>(y) + i;
            const u4v w = __builtin_bit_cast(u4v, h);
            if constexpr (NT) __builtin_nontemporal_store(w, p);
            else *p = w;
        }
    }
}

template <int FMT, int YDT>
static void launch_dq(const uint8_t *q, const uint8_t *scale, int64_t elems, void *y,
                      hipStream_t stream) {
    const int64_t n = elems / Vec<YDT>::n, blocks = (n + 1023) / 1024;
    const dim3 grid((unsigned)(blocks < 4096 ? blocks : 4096));
    if (elems * dt_bytes(YDT) > kNtLoadBytes)
        mx_dequant_kernel<FMT, YDT, true><<<grid, 256, 0, stream>>>(q, scale, n, y);
    else
        mx_dequant_kernel<FMT, YDT, false><<<grid, 256, 0, stream>>>(q, scale, n, y);
}

void launch_dequant_mx(const uint8_t *q, const uint8_t *scale, int fmt, int64_t rows, int64_t K,
                       void *y, int y_dt, hipStream_t stream) {
    const int64_t n = rows * K;
    if (fmt == E2M1) {
        if (y_dt == F32) launch_dq<E2M1, F32>(q, scale, n, y, stream);
        else if (y_dt == F16) launch_dq<E2M1, F16>(q, scale, n, y, stream);
        else launch_dq<E2M1, BF16>(q, scale, n, y, stream);
    } else {
        if (y_dt == F32) launch_dq<E4M3, F32>(q, scale, n, y, stream);
        else if (y_dt == F16) launch_dq<E4M3, F16>(q, scale, n, y, stream);
        else launch_dq<E4M3, BF16>(q, scale, n, y, stream);
    }
}

}  // namespace sq
