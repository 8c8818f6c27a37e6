// Rotary positions with the quantized write of keys and values into the
// microscaled cache, and the way back (include/sq_kv.h).
//
// Both are one pass over their data, eight elements a lane and four lanes (a
// quad) a block of 32, as the row quantizer.  A block of 256 threads takes 256
// lanes' worth of tokens, one head's row of each at a time: a page holds a
// head's tokens next to one another, so the short rows of codes (64 bytes of
// e2m1 for 128 channels) fill whole cache lines.  Rows are loaded four ahead.
// With few tokens a block takes fewer of them and several heads at a time, and
// the heads are dealt to blocks of their own.
#include "kv_device.h"

namespace sq {

constexpr int kAhead = 4;

// Tokens of a block (a power of two) and blocks along the heads' rows.
struct Deal {
    int tok_log;
    int64_t groups, y;
};
static Deal deal_rows(int64_t tokens, int dim, int rows, int most_log) {
    Deal d = {};
    const int all = 256 / (dim / 8);  // 32, 16 or 8
    // (as many tokens at a time as still make 1024 blocks with all heads apart)
    int log = 0;
    while (log < most_log && 2 << log <= all && (tokens >> (log + 1)) * rows >= 1024) ++log;
    d.tok_log = log;
    d.groups = (tokens + (1 << log) - 1) >> log;
    const int64_t at_once = all >> log, most = (rows + at_once - 1) / at_once;
    // enough blocks to fill the GPU, and no more: each forms its tokens' angles
    const int64_t want = (1024 + d.groups - 1) / d.groups;
    d.y = want < most ? want : most;
    return d;
}

// ---------------------------------------------------------- rotary and write

// The angles are formed, and their sine and cosine taken, in 64 bits once for
// a token and pair, and shared by its heads through LDS: at position 10^5 an
// fp32 product p * f is off by up to 2^-8 of a radian.
template <int DT, int FMT, bool NT>
__global__ __launch_bounds__(256) void kv_write_kernel(const RopeWrite a, int tok_log) {
    __shared__ float s_cos[1024], s_sin[1024];  // [tokens][rotary / 2] (256 / (D / 8) D / 2 = 1024)
    const int tid = threadIdx.x, tok = 1 << tok_log;
    const int64_t t0 = (int64_t)blockIdx.x << tok_log;
    const int half = a.rotary >> 1;
    for (int i = tid; i < tok * half; i += 256) {
        const int tb = i / half, f = i - tb * half;
        if (t0 + tb < a.T) {
            const double ang = (double)a.positions[t0 + tb] * a.inv_freq[f];
            double sn, cn;
            sincos(ang, &sn, &cn);
            s_cos[i] = (float)(cn * a.amplitude);
            s_sin[i] = (float)(sn * a.amplitude);
        }
    }
    __syncthreads();
    const int d8_log = 31 - __builtin_clz(a.cache.dim >> 3), d8 = 1 << d8_log;  // lanes of a row
    const int rows = a.q_heads + 2 * a.cache.heads;
    const int64_t slots = a.cache.pages << a.cache.page_log;
    const int c = tid & (d8 - 1), tb = (tid >> d8_log) & (tok - 1);
    const int64_t t = t0 + tb;
    if (t >= a.T) return;  // (a whole row of lanes)
    const int64_t slot = a.slots[t];
    const bool stored = slot >= 0 && slot < slots;
    const int64_t page = slot >> a.cache.page_log;
    const int at = (int)(slot & ((1 << a.cache.page_log) - 1));
    const int e0 = c * 8;
    const bool turned = e0 < a.rotary, low = e0 < half;
    // the other half of a pair, and the pairs' angles
    const int other = a.layout ? c : low ? c + (half >> 3) : c - (half >> 3);
    const int f0 = tb * half + (a.layout ? e0 >> 1 : low ? e0 : e0 - half);
    const int at_once = 256 >> (d8_log + tok_log), step = at_once * gridDim.y;
    for (int r0 = blockIdx.y * at_once + (tid >> (d8_log + tok_log)); r0 < rows; r0 += kAhead * step) {
        Raw8<DT> raw[kAhead], pair[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            // rows: the queries' heads, the keys', the values' (past the last: it again)
            int r = r0 + u * step;
            r = r < rows ? r : r0;
            const int k = r - a.q_heads, v = k - a.cache.heads;
            const char *x = r < a.q_heads         ? (const char *)a.q + (t * a.q_st + r * a.q_sh) * dt_bytes(DT)
                            : v < 0 ? (const char *)a.k + (t * a.k_st + k * a.k_sh) * dt_bytes(DT)
                                    : (const char *)a.v + (t * a.v_st + v * a.v_sh) * dt_bytes(DT);
            raw[u] = load8<DT, NT>(x, c);
            if (turned && v < 0 && a.layout == 0) pair[u] = load8<DT, NT>(x, other);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int r = r0 + u * step;
            if (r >= rows) break;
            const bool is_q = r < a.q_heads, is_k = !is_q && r < a.q_heads + a.cache.heads;
            const int h = is_q ? r : is_k ? r - a.q_heads : r - a.q_heads - a.cache.heads;
            float v[8];
            widen8<DT>(raw[u], v);
            if ((is_q || is_k) && turned) {
                if (a.layout == 0) {
                    float o[8];
                    widen8<DT>(pair[u], o);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float p = v[i] * s_cos[f0 + i], s = o[i] * s_sin[f0 + i];
                        v[i] = low ? p - s : p + s;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float co = s_cos[f0 + i], si = s_sin[f0 + i];
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
                constexpr int W = DT == F32 ? 2 : 1;
                T out[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) out[i] = narrow<DT>(v[i]);
                u4v *p = reinterpret_cast<u4v *>(a.q_out) + ((((t * a.q_heads + h) << d8_log) + c)) * W;
                const Raw8<DT> w = __builtin_bit_cast(Raw8<DT>, out);
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    if constexpr (NT) __builtin_nontemporal_store(__builtin_bit_cast(u4v, w.v[i]), p + i);
                    else p[i] = __builtin_bit_cast(u4v, w.v[i]);
                }
            } else {
                uint32_t e;
                const MxCodes<FMT> code = mx_encode8<FMT>(v, e);
                if (stored)
                    mx_store8<FMT, false>(is_k ? a.cache.kq : a.cache.vq, is_k ? a.cache.ks : a.cache.vs,
                                          (kv_row(a.cache, page, h, at) << d8_log) + c, code, e);
            }
        }
    }
}

template <int DT, int FMT>
static void launch_write_fmt(const RopeWrite &a, hipStream_t stream) {
    const int rows = a.q_heads + 2 * a.cache.heads;
    // (four tokens at the most: 16384 tokens of 64 + 2 x 8 heads of 128 in bf16
    // 130 us, 622 MB at 4.8 TB/s; with one 135, eight 141, sixteen 157, whose
    // pieces of 256 bytes of a token lie far apart in time; fp32 rows 325 us, 1.23
    // GB at 3.8 TB/s, to e4m3 330)
    const Deal d = deal_rows(a.T, a.cache.dim, rows, 2);
    const dim3 grid((unsigned)d.groups, (unsigned)d.y);
    // (past what the caches hold, data read once is kept out of them: 129 us for
    // the 16384 tokens above, 135 without; 333 tokens either way 9)
    if (a.T * rows * a.cache.dim * dt_bytes(DT) > kNtLoadBytes)
        kv_write_kernel<DT, FMT, true><<<grid, 256, 0, stream>>>(a, d.tok_log);
    else
        kv_write_kernel<DT, FMT, false><<<grid, 256, 0, stream>>>(a, d.tok_log);
}

template <int DT>
static void launch_write_dt(const RopeWrite &a, hipStream_t stream) {
    if (a.cache.fmt == E2M1) launch_write_fmt<DT, E2M1>(a, stream);
    else launch_write_fmt<DT, E4M3>(a, stream);
}

void launch_rope_write(const RopeWrite &a, int dt, hipStream_t stream) {
    if (dt == F32) launch_write_dt<F32>(a, stream);
    else if (dt == F16) launch_write_dt<F16>(a, stream);
    else launch_write_dt<BF16>(a, stream);
}

// -------------------------------------------------------------- the way back

// Bound by memory: 62494 tokens of 8 heads of 128 from e2m1 to bf16 50 us, 324 MB
// at 6.5 TB/s; from e4m3 71 us, 388 MB at 5.5.  To fp32, where each of a lane's two
// stores fills half of every 32 bytes, 204 .. 241 us (580 MB) and 214 (644 MB).

// Two fp32 values of a byte of e2m1 codes, or of a half of e4m3 codes.
template <int FMT>
__device__ __forceinline__ void widen_codes8(const uint32_t *w, float s, float (&v)[8]) {
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
}

template <int DT, int FMT, bool NT>
__global__ __launch_bounds__(256) void kv_read_kernel(const KvRead a, int tok_log) {
    const int tid = threadIdx.x, tok = 1 << tok_log;
    const int d8_log = 31 - __builtin_clz(a.cache.dim >> 3), d8 = 1 << d8_log;
    const int c = tid & (d8 - 1), tb = (tid >> d8_log) & (tok - 1);
    const int64_t row = ((int64_t)blockIdx.x << tok_log) + tb;
    if (row >= a.total || row >= a.cu[a.B] || row < a.cu[0]) return;
    const int b = kv_find(a.cu, a.B, row);
    const int64_t t = row - a.cu[b], col = t >> a.cache.page_log;
    int64_t page = t >= 0 && col < a.width ? a.table[b * a.width + col] : -1;
    const bool held = page >= 0 && page < a.cache.pages;
    page = held ? page : 0;
    const uint32_t nan = held ? 0u : 255u;
    const int at = (int)(t & ((1 << a.cache.page_log) - 1));
    const int rows = 2 * a.cache.heads;  // the keys' heads, the values'
    const int at_once = 256 >> (d8_log + tok_log), step = at_once * gridDim.y;
    for (int r0 = blockIdx.y * at_once + (tid >> (d8_log + tok_log)); r0 < rows; r0 += kAhead * step) {
        uint32_t w[kAhead][2], e[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            int r = r0 + u * step;
            r = r < rows ? r : r0;
            const bool is_k = r < a.cache.heads;
            const int64_t i = (kv_row(a.cache, page, is_k ? r : r - a.cache.heads, at) << d8_log) + c;
            const uint8_t *q = is_k ? a.cache.kq : a.cache.vq;
            if constexpr (FMT == E2M1) {
                w[u][0] = reinterpret_cast<const uint32_t *>(q)[i];
            } else {
                const uint2 x = reinterpret_cast<const uint2 *>(q)[i];
                w[u][0] = x.x;
                w[u][1] = x.y;
            }
            e[u] = (is_k ? a.cache.ks : a.cache.vs)[i >> 2];
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int r = r0 + u * step;
            if (r >= rows) break;
            const bool is_k = r < a.cache.heads;
            const float s = e8m0(e[u] | nan);
            constexpr int W = DT == F32 ? 2 : 1;
            u4v *dst = reinterpret_cast<u4v *>(is_k ? a.k : a.v) +
                       (((row * a.cache.heads + (is_k ? r : r - a.cache.heads)) << d8_log) + c) * W;
            u4v out[W];
            if constexpr (DT == F32) {
                float v[8];
                widen_codes8<FMT>(w[u], s, v);
                out[0] = __builtin_bit_cast(u4v, make_float4(v[0], v[1], v[2], v[3]));
                out[1] = __builtin_bit_cast(u4v, make_float4(v[4], v[5], v[6], v[7]));
            } else {
                out[0] = __builtin_bit_cast(u4v, codes8_to_16<FMT, DT>(w[u], s));
            }
#pragma unroll
            for (int i = 0; i < W; ++i) {
                if constexpr (NT) __builtin_nontemporal_store(out[i], dst + i);
                else dst[i] = out[i];
            }
        }
    }
}

template <int DT, int FMT>
static void launch_read_fmt(const KvRead &a, hipStream_t stream) {
    const int rows = 2 * a.cache.heads;
    const Deal d = deal_rows(a.total, a.cache.dim, rows, 5);
    const dim3 grid((unsigned)d.groups, (unsigned)d.y);
    // (as above: 51 us for 62494 tokens, 63 without)
    if (a.total * rows * a.cache.dim * dt_bytes(DT) > kNtLoadBytes)
        kv_read_kernel<DT, FMT, true><<<grid, 256, 0, stream>>>(a, d.tok_log);
    else
        kv_read_kernel<DT, FMT, false><<<grid, 256, 0, stream>>>(a, d.tok_log);
}

template <int DT>
static void launch_read_dt(const KvRead &a, hipStream_t stream) {
    if (a.cache.fmt == E2M1) launch_read_fmt<DT, E2M1>(a, stream);
    else launch_read_fmt<DT, E4M3>(a, stream);
}

void launch_kv_read(const KvRead &a, int dt, hipStream_t stream) {
    if (dt == F32) launch_read_dt<F32>(a, stream);
    else if (dt == F16) launch_read_dt<F16>(a, stream);
    else launch_read_dt<BF16>(a, stream);
}

}  // namespace sq
