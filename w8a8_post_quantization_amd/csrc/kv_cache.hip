// Rotary positions with the quantized write of keys and values into the
// microscaled cache, and the way back (include/sq_kv.h).
//
// Both are one pass over their data, eight elements a lane and four lanes (a
// quad) a block of 32, as the row quantizer.  A block of threads takes kTok
// successive tokens, neighbouring lanes a head's row, then the same head of the
// next token: a page holds a head's tokens next to one another, so the short
// rows of codes (64 bytes of e2m1 for 128 channels) fill whole cache lines.
#include "kv_device.h"

namespace sq {

constexpr int kTok = 4;

// ---------------------------------------------------------- rotary and write

// The angles are formed, and their sine and cosine taken, in 64 bits once for
// a token and pair, and shared by its heads through LDS: at position 10^5 an
// fp32 product p * f is off by up to 2^-8 of a radian.
template <int DT, int FMT>
__global__ __launch_bounds__(256) void kv_write_kernel(const RopeWrite a) {
    __shared__ float cs[kTok][2][128];
    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * kTok;
    const int half = a.rotary >> 1;
    for (int i = tid; i < kTok * half; i += 256) {
        const int tb = i / half, f = i - tb * half;
        if (t0 + tb < a.T) {
            const double ang = (double)a.positions[t0 + tb] * a.inv_freq[f];
            double sn, cn;
            sincos(ang, &sn, &cn);
            cs[tb][0][f] = (float)(cn * a.amplitude);
            cs[tb][1][f] = (float)(sn * a.amplitude);
        }
    }
    __syncthreads();
    const int d8 = a.cache.dim >> 3;  // lanes of a row: 8, 16 or 32
    const int rows = a.q_heads + 2 * a.cache.heads;
    const int64_t slots = a.cache.pages << a.cache.page_log;
    const int c = tid % d8, tb = tid / d8 % kTok;
    const int64_t t = t0 + tb;
    if (t >= a.T) return;  // (a whole row of lanes)
    const int64_t slot = a.slots[t];
    const bool stored = slot >= 0 && slot < slots;
    const int e0 = c * 8;
    const int step = 256 / (d8 * kTok) * gridDim.y;
    for (int r = blockIdx.y * (256 / (d8 * kTok)) + tid / (d8 * kTok); r < rows; r += step) {
        // rows: the queries' heads, the keys', the values'
        const bool is_q = r < a.q_heads;
        const bool is_k = !is_q && r < a.q_heads + a.cache.heads;
        const int h = is_q ? r : is_k ? r - a.q_heads : r - a.q_heads - a.cache.heads;
        const char *x = is_q   ? (const char *)a.q + (t * a.q_st + h * a.q_sh) * dt_bytes(DT)
                        : is_k ? (const char *)a.k + (t * a.k_st + h * a.k_sh) * dt_bytes(DT)
                               : (const char *)a.v + (t * a.v_st + h * a.v_sh) * dt_bytes(DT);
        float v[8];
        widen8<DT>(load8<DT, false>(x, c), v);
        if ((is_q || is_k) && e0 < a.rotary) {
            if (a.layout == 0) {
                const bool low = e0 < half;
                float o[8];
                widen8<DT>(load8<DT, false>(x, low ? c + (half >> 3) : c - (half >> 3)), o);
                const int f = low ? e0 : e0 - half;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p = v[i] * cs[tb][0][f + i], s = o[i] * cs[tb][1][f + i];
                    v[i] = low ? p - s : p + s;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float co = cs[tb][0][(e0 >> 1) + i], si = cs[tb][1][(e0 >> 1) + i];
                    const float x1 = v[2 * i], x2 = v[2 * i + 1];
                    const float p1 = x1 * co, p2 = x2 * si, p3 = x2 * co, p4 = x1 * si;
                    v[2 * i] = p1 - p2;
                    v[2 * i + 1] = p3 + p4;
                }
            }
        }
        const float *mul = is_q ? a.q_mul : is_k ? a.k_mul : nullptr;
        if (mul) {
            float m[8];
            load_f32x8(mul + (int64_t)h * a.cache.dim + e0, m);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = v[i] * m[i];
        }
        if (is_q) {
            using T = typename OutT<DT>::T;
            T out[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) out[i] = narrow<DT>(v[i]);
            u4v *p = reinterpret_cast<u4v *>(a.q_out) +
                     ((t * a.q_heads + h) * d8 + c) * (DT == F32 ? 2 : 1);
            const Raw8<DT> w = __builtin_bit_cast(Raw8<DT>, out);
#pragma unroll
            for (int i = 0; i < (DT == F32 ? 2 : 1); ++i)
                p[i] = __builtin_bit_cast(u4v, w.v[i]);
        } else {
            uint32_t e;
            const MxCodes<FMT> code = mx_encode8<FMT>(v, e);
            if (stored) {
                const int64_t row = kv_row(a.cache, slot >> a.cache.page_log, h,
                                           (int)(slot & ((1 << a.cache.page_log) - 1)));
                mx_store8<FMT, false>(is_k ? a.cache.kq : a.cache.vq, is_k ? a.cache.ks : a.cache.vs,
                                      row * d8 + c, code, e);
            }
        }
    }
}

template <int DT>
static void launch_write_dt(const RopeWrite &a, hipStream_t stream) {
    const int64_t groups = (a.T + kTok - 1) / kTok;
    // rows that a block takes at a time; with few tokens the rows are spread
    // over blocks of their own
    const int per = 256 / ((a.cache.dim >> 3) * kTok);
    const int rows = a.q_heads + 2 * a.cache.heads;
    int64_t y = (rows + per - 1) / per;
    const int64_t most = 1024 / groups > 1 ? 1024 / groups : 1;
    y = y < most ? y : most;
    const dim3 grid((unsigned)groups, (unsigned)y);
    if (a.cache.fmt == E2M1) kv_write_kernel<DT, E2M1><<<grid, 256, 0, stream>>>(a);
    else kv_write_kernel<DT, E4M3><<<grid, 256, 0, stream>>>(a);
}

void launch_rope_write(const RopeWrite &a, int dt, hipStream_t stream) {
    if (dt == F32) launch_write_dt<F32>(a, stream);
    else if (dt == F16) launch_write_dt<F16>(a, stream);
    else launch_write_dt<BF16>(a, stream);
}

// -------------------------------------------------------------- the way back

template <int DT, int FMT>
__global__ __launch_bounds__(256) void kv_read_kernel(const KvRead a) {
    const int tid = threadIdx.x, d8 = a.cache.dim >> 3;
    const int c = tid % d8, tb = tid / d8 % kTok;
    const int64_t row = (int64_t)blockIdx.x * kTok + tb;
    if (row >= a.total || row >= a.cu[a.B] || row < a.cu[0]) return;
    const int b = kv_find(a.cu, a.B, row);
    const int64_t t = row - a.cu[b], col = t >> a.cache.page_log;
    int64_t page = t >= 0 && col < a.width ? a.table[b * a.width + col] : -1;
    const bool held = page >= 0 && page < a.cache.pages;
    page = held ? page : 0;
    const int at = (int)(t & ((1 << a.cache.page_log) - 1));
    const int rows = 2 * a.cache.heads;  // the keys' heads, the values'
    const int step = 256 / (d8 * kTok) * gridDim.y;
    for (int r = blockIdx.y * (256 / (d8 * kTok)) + tid / (d8 * kTok); r < rows; r += step) {
        const bool is_k = r < a.cache.heads;
        const int h = is_k ? r : r - a.cache.heads;
        const int64_t i = kv_row(a.cache, page, h, at) * d8 + c;
        const uint8_t *q = is_k ? a.cache.kq : a.cache.vq;
        uint32_t w[2];
        if constexpr (FMT == E2M1) {
            w[0] = reinterpret_cast<const uint32_t *>(q)[i];
        } else {
            const uint2 u = reinterpret_cast<const uint2 *>(q)[i];
            w[0] = u.x;
            w[1] = u.y;
        }
        const uint32_t e = held ? (is_k ? a.cache.ks : a.cache.vs)[i >> 2] : 255u;
        void *y = is_k ? a.k : a.v;
        const int64_t o = (row * a.cache.heads + h) * d8 + c;
        if constexpr (DT == F32) {
            // (bf16 would lose e4m3 blocks of the smallest scales: widened on
            // its own)
            float v[8];
            const float s = e8m0(e);
            f32x2 p[4];
            if constexpr (FMT == E2M1) {
                p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], s, 0);
                p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], s, 1);
                p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], s, 2);
                p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], s, 3);
            } else {
                p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[0], s, false);
                p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[0], s, true);
                p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[1], s, false);
                p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[1], s, true);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[2 * k] = p[k][0];
                v[2 * k + 1] = p[k][1];
            }
            u4v *dst = reinterpret_cast<u4v *>(y) + 2 * o;
            dst[0] = __builtin_bit_cast(u4v, make_float4(v[0], v[1], v[2], v[3]));
            dst[1] = __builtin_bit_cast(u4v, make_float4(v[4], v[5], v[6], v[7]));
        } else {
            reinterpret_cast<u4v *>(y)[o] = __builtin_bit_cast(u4v, codes8_to_16<FMT, DT>(w, e8m0(e)));
        }
    }
}

template <int DT>
static void launch_read_dt(const KvRead &a, hipStream_t stream) {
    const int64_t groups = (a.total + kTok - 1) / kTok;
    const int per = 256 / ((a.cache.dim >> 3) * kTok);
    int64_t y = (2 * a.cache.heads + per - 1) / per;
    const int64_t most = 1024 / groups > 1 ? 1024 / groups : 1;
    y = y < most ? y : most;
    const dim3 grid((unsigned)groups, (unsigned)y);
    if (a.cache.fmt == E2M1) kv_read_kernel<DT, E2M1><<<grid, 256, 0, stream>>>(a);
    else kv_read_kernel<DT, E4M3><<<grid, 256, 0, stream>>>(a);
}

void launch_kv_read(const KvRead &a, int dt, hipStream_t stream) {
    if (dt == F32) launch_read_dt<F32>(a, stream);
    else if (dt == F16) launch_read_dt<F16>(a, stream);
    else launch_read_dt<BF16>(a, stream);
}

}  // namespace sq
