// Attention over the microscaled cache, many queries a sequence (include/
// sq_kv.h): kv_attn.hip's arithmetic and orientation with matrix instructions
// of 32 x 32 x 16, and the keys and values of a tile converted once for a
// block and shared through LDS.
//
// A block takes 128 WR rows (a row: a query of one of the heads that share the
// key head), 32 WR a wave, over its keys in tiles of 64.  In LDS keys lie
// [key][channel], values [channel][key], both so that an operand is one
// 16-byte read; the values' keys are in the order in which the weights lie in
// the lanes.  Chunks of 16 bytes are exchanged by an xor with the row's number,
// so that the lanes of a read take all banks.
#include "kv_attn_device.h"

namespace sq {

constexpr int kKeys = 64;

// Where chunk `ch` (16 bytes) of key `key`, and of channel `d`, lies in LDS.
template <int D>
__device__ __forceinline__ int key_chunk(int key, int ch) { return key * (D / 8) + (ch ^ (key & 7)); }
__device__ __forceinline__ int value_chunk(int d, int ch) { return d * (kKeys / 8) + (ch ^ ((d ^ d >> 3) & 7)); }

template <int D, int FMT, int DT, int WR>
__global__ __launch_bounds__(256) void kv_tile_kernel(const KvAttention a, int rows_min, int splits, float *parts) {
    constexpr int NB = D / 32, J = D / 16, S = D / 16, JT = D / 32, R = 128 * WR;
    constexpr int RB = FMT == E2M1 ? D / 2 : D;
    constexpr int KN = NB * (FMT == E2M1 ? 4 : 8);     // code bytes of a key, a quarter of its channels
    constexpr int KS = NB < 4 ? 1 : NB / 4;            // scale bytes of those
    constexpr int VN = FMT == E2M1 ? D / 32 : D / 16;  // code bytes of a value, a sixteenth of its channels
    __shared__ uint4 s_k[kKeys * D / 8], s_v[kKeys * D / 8];
    __shared__ int s_pre[257], s_at[2], s_bad[2];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n32 = lane & 31, hh = lane >> 5;
    const int heads = a.cache.heads, plog = a.cache.page_log, group = a.group;

    // The block's rows: tiles of all long sequences in a row, the last (with the
    // most keys) first.
    const auto tiles_of = [&](const KvSeq &s) -> int {
        const int64_t rows = (int64_t)s.nq * group;
        return rows < rows_min ? 0 : (int)((rows + R - 1) / R);
    };
    const int per_thread = (a.B + 255) / 256;
    const int b_first = tid * per_thread;
    {
        int sum = 0;
        for (int i = 0; i < per_thread && b_first + i < a.B; ++i) sum += tiles_of(kv_seq(a, b_first + i));
        s_pre[tid + 1] = sum;
        if (tid == 0) s_pre[0] = 0;
        __syncthreads();
        for (int off = 1; off < 256; off <<= 1) {
            const int v = tid >= off ? s_pre[tid + 1 - off] : 0;
            __syncthreads();
            s_pre[tid + 1] += v;
            __syncthreads();
        }
    }
    const int want = s_pre[256] - 1 - (int)(blockIdx.x / heads);
    if (want < 0) return;
    if (s_pre[tid] <= want && want < s_pre[tid + 1]) {
        int before = s_pre[tid], b = b_first;
        for (;;) {
            const int n = tiles_of(kv_seq(a, b));
            if (want < before + n) break;
            before += n;
            ++b;
        }
        s_at[0] = b;
        s_at[1] = want - before;
    }
    __syncthreads();
    const int b = __builtin_amdgcn_readfirstlane(s_at[0]);
    const int tile = __builtin_amdgcn_readfirstlane(s_at[1]);
    const int h = blockIdx.x % heads, split = blockIdx.y;
    const KvSeq seq = kv_seq(a, b);
    const int rows = seq.nq * group;  // (T * q_heads < 2^31)

    // Keys that the rows from r to e - 1 see: all of them, any of them.
    const auto span = [&](int r, int e, int &all_lo, int &all_hi, int &any_lo, int &any_hi) {
        const int p0 = seq.nk - seq.nq + r / group, p1 = seq.nk - seq.nq + (e - 1) / group;
        any_hi = a.causal ? (p1 + 1 > 0 ? p1 + 1 : 0) : seq.nk;
        all_hi = a.causal ? p0 + 1 : seq.nk;
        any_lo = a.window && (int64_t)p0 - a.window + 1 > 0 ? (int)(p0 - a.window + 1) : 0;
        all_lo = a.window && (int64_t)p1 - a.window + 1 > 0 ? (int)(p1 - a.window + 1) : 0;
    };
    const int r_first = tile * R, r_end = r_first + R < rows ? r_first + R : rows;
    int t_all_lo, t_all_hi, t_lo, t_hi;
    span(r_first, r_end, t_all_lo, t_all_hi, t_lo, t_hi);
    const int w_first = r_first + wave * 32 * WR;
    const int w_end = w_first + 32 * WR < rows ? w_first + 32 * WR : rows;
    int w_all_lo = 0, w_all_hi = 0, w_lo = 0, w_hi = 0;
    if (w_first < rows) span(w_first, w_end, w_all_lo, w_all_hi, w_lo, w_hi);

    uint4 qf[WR][S];
    int r_lo[WR], r_hi[WR];
#pragma unroll
    for (int wr = 0; wr < WR; ++wr) {
        const int r = w_first + wr * 32 + n32;
        const int i = r / group;
        const char *x = (const char *)a.q +
                        ((int64_t)(seq.q0 + i) * a.q_st + (int64_t)(h * group + r - i * group) * a.q_sh) * 2;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            qf[wr][s] = make_uint4(0, 0, 0, 0);
            if (r < rows) qf[wr][s] = reinterpret_cast<const uint4 *>(x)[2 * s + hh];
        }
        const int p = seq.nk - seq.nq + i;
        r_hi[wr] = r < rows ? (a.causal ? p + 1 : seq.nk) : 0;
        r_lo[wr] = a.window && (int64_t)p - a.window + 1 > 0 ? (int)(p - a.window + 1) : 0;
    }

    float m[WR], l[WR];
    f32x16 o[WR][JT];
#pragma unroll
    for (int wr = 0; wr < WR; ++wr) {
        m[wr] = kNoMax;
        l[wr] = 0.0f;
#pragma unroll
        for (int j = 0; j < JT; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[wr][j][i] = 0.0f;
    }

    // The split's tiles of keys.
    const int t_base = t_lo & ~(kKeys - 1);
    const int n_tiles = t_hi > t_lo ? (t_hi - t_base + kKeys - 1) / kKeys : 0;
    const int k0 = (int)((int64_t)n_tiles * split / splits), k1 = (int)((int64_t)n_tiles * (split + 1) / splits);
    const float c = a.scale * 1.44269504088896341f;
    const int32_t *const table = a.table + (int64_t)b * a.width;
    const int g_last = (t_hi - 1) >> 4;

    // As a thread stages a tile: a quarter of one key's channels, and of four
    // successive keys a sixteenth of the values' channels.
    const int sk = tid >> 2, sc = tid & 3, sq4 = tid >> 4, sn = tid & 15;
    Words<KN> rk;
    uint32_t rks[KS];
    Words<VN> rv[4];
    uint32_t rvs[4];
    const auto place = [&](int key, int64_t &row) -> bool {
        int grp = key >> 4;
        grp = grp < g_last ? grp : g_last;
        int64_t page = table[grp >> (plog - 4)];
        const bool held = page >= 0 && page < a.cache.pages;
        page = held ? page : 0;
        row = kv_row(a.cache, page, h, ((grp & ((1 << (plog - 4)) - 1)) << 4) + (key & 15));
        return held;
    };
    const auto load = [&](int t) {
        int64_t row;
        bool held = place(t + sk, row);
        rk = load_codes<KN>(a.cache.kq + row * RB + sc * KN);
#pragma unroll
        for (int i = 0; i < KS; ++i) rks[i] = held ? a.cache.ks[row * NB + sc * NB / 4 + i] : 255u;
        held = place(t + 4 * sq4, row);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rv[i] = load_codes<VN>(a.cache.vq + (row + i) * RB + sn * VN);
            rvs[i] = held ? a.cache.vs[(row + i) * NB + sn * NB / 16] : 255u;
        }
    };
    const auto stage = [&](int t, int turn) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const float s = e8m0(rks[NB < 4 ? 0 : i / 4]);
            s_k[key_chunk<D>(sk, sc * NB + i)] =
                codes8_to_16<FMT, DT>(&rk.w[i * (FMT == E2M1 ? 1 : 2)], s);
        }
        const bool masked = t < t_all_lo || t + kKeys > t_all_hi;
        if (masked) {
            // keys that no row of the block sees are taken as 0: what their
            // place holds may be anything
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = t + 4 * sq4 + i;
                if (key < t_lo || key >= t_hi) {
                    rv[i] = Words<VN>{};
                    rvs[i] = 0;
                }
            }
        }
        // a quad of keys in its group of 16: quads 0, 2, 1, 3
        const int half = (sq4 & 3) >> 1, ch = (sq4 >> 2) * 2 + (sq4 & 1);
        uint32_t bad = 0;
#pragma unroll
        for (int q = 0; q < J / 2; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pair_of<FMT, DT>(rv[i], q, e8m0(rvs[i]));
            if (masked) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t up, down;
                    split_nonfinite<DT>(w[i], up, down);
                    bad |= up | down;
                }
            }
#pragma unroll
            for (int odd = 0; odd < 2; ++odd) {
                const uint32_t sel = odd ? 0x07060302u : 0x05040100u;
                reinterpret_cast<uint2 *>(s_v)[2 * value_chunk(sn * J + 2 * q + odd, ch) + half] =
                    make_uint2(__builtin_amdgcn_perm(w[1], w[0], sel), __builtin_amdgcn_perm(w[3], w[2], sel));
            }
        }
        if (bad) s_bad[turn] = 1;
    };

    if (k0 < k1) load(t_base + k0 * kKeys);
    if (tid == 0) s_bad[k0 & 1] = 0;
    for (int k = k0; k < k1; ++k) {
        const int t0 = t_base + k * kKeys;
        __syncthreads();
        stage(t0, k & 1);
        if (tid == 0) s_bad[~k & 1] = 0;
        __syncthreads();
        const bool bad = __builtin_amdgcn_readfirstlane(s_bad[k & 1]) != 0;
        if (k + 1 < k1) load(t0 + kKeys);
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
            const int t = t0 + 32 * sub;
            if (t >= w_hi || t + 32 <= w_lo) continue;  // no row of the wave sees any
            f32x16 st[WR];
#pragma unroll
            for (int wr = 0; wr < WR; ++wr)
#pragma unroll
                for (int i = 0; i < 16; ++i) st[wr][i] = 0.0f;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const uint4 kf = s_k[key_chunk<D>(32 * sub + n32, 2 * s + hh)];
#pragma unroll
                for (int wr = 0; wr < WR; ++wr) st[wr] = mfma32<DT>(kf, qf[wr][s], st[wr]);
            }
            const bool masked = t < w_all_lo || t + 32 > w_all_hi;
            uint4 pf[WR][2], seen[WR][2];
#pragma unroll
            for (int wr = 0; wr < WR; ++wr) {
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < 16; ++i) st[wr][i] *= c;
                if (masked) {
                    uint32_t v[8] = {};
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int key = t + (i & 3) + 8 * (i >> 2) + 4 * hh;
                        const bool vis = key >= r_lo[wr] && key < r_hi[wr];
                        st[wr][i] = vis ? st[wr][i] : -INFINITY;
                        v[i >> 1] |= vis ? (DT == BF16 ? 0x3f80u : 0x3c00u) << (16 * (i & 1)) : 0u;
                    }
                    seen[wr][0] = make_uint4(v[0], v[1], v[2], v[3]);
                    seen[wr][1] = make_uint4(v[4], v[5], v[6], v[7]);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, st[wr][i]);
                // (the maximum may trail by 8, as in kv_attn.hip)
                if (__any(top > m[wr] + 8.0f)) {
                    top = fmaxf(top, __shfl_xor(top, 32, 64));
                    const float mn = fmaxf(m[wr], top);
                    const float f = __builtin_amdgcn_exp2f(m[wr] - mn);
                    m[wr] = mn;
                    l[wr] *= f;
#pragma unroll
                    for (int j = 0; j < JT; ++j) o[wr][j] *= f;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    st[wr][i] = __builtin_amdgcn_exp2f(st[wr][i] - m[wr]);
                    l[wr] += st[wr][i];
                }
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    pf[wr][u] = make_uint4(pack16<DT>(st[wr][8 * u], st[wr][8 * u + 1]),
                                           pack16<DT>(st[wr][8 * u + 2], st[wr][8 * u + 3]),
                                           pack16<DT>(st[wr][8 * u + 4], st[wr][8 * u + 5]),
                                           pack16<DT>(st[wr][8 * u + 6], st[wr][8 * u + 7]));
            }
#pragma unroll
            for (int j = 0; j < JT; ++j)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint4 vf = s_v[value_chunk(32 * j + n32, 4 * sub + 2 * u + hh)];
                    if (bad) {
                        // (as in kv_attn.hip: a weight of 0 would not keep them out)
                        uint4 up, down;
                        vf.x = split_nonfinite<DT>(vf.x, up.x, down.x);
                        vf.y = split_nonfinite<DT>(vf.y, up.y, down.y);
                        vf.z = split_nonfinite<DT>(vf.z, up.z, down.z);
                        vf.w = split_nonfinite<DT>(vf.w, up.w, down.w);
#pragma unroll
                        for (int wr = 0; wr < WR; ++wr) {
                            const uint32_t one = DT == BF16 ? 0x3f803f80u : 0x3c003c00u;
                            const uint4 see = masked ? seen[wr][u] : make_uint4(one, one, one, one);
                            f32x16 z;
#pragma unroll
                            for (int i = 0; i < 16; ++i) z[i] = 0.0f;
                            const f32x16 cu = mfma32<DT>(up, see, z);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (cu[i] > 0) o[wr][j][i] += INFINITY;
                            const f32x16 cd = mfma32<DT>(down, see, z);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (cd[i] > 0) o[wr][j][i] -= INFINITY;
                        }
                    }
#pragma unroll
                    for (int wr = 0; wr < WR; ++wr) o[wr][j] = mfma32<DT>(vf, pf[wr][u], o[wr][j]);
                }
        }
    }

#pragma unroll
    for (int wr = 0; wr < WR; ++wr) {
        const int r = w_first + wr * 32 + n32;
        l[wr] += __shfl_xor(l[wr], 32, 64);
        if (r >= rows) continue;
        const int i = r / group;
        const int64_t row = (int64_t)(seq.q0 + i) * a.q_heads + h * group + r - i * group;
        if (splits == 1) {
            const float inv = row_factor(l[wr], seq.over);
            uint2 *y = reinterpret_cast<uint2 *>(a.y) + row * (D / 4) + hh;
#pragma unroll
            for (int j = 0; j < JT; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    y[8 * j + 2 * k] = make_uint2(pack16<DT>(o[wr][j][4 * k] * inv, o[wr][j][4 * k + 1] * inv),
                                                  pack16<DT>(o[wr][j][4 * k + 2] * inv, o[wr][j][4 * k + 3] * inv));
        } else {
            // values of all rows and splits, then their maxima and sums
            const int64_t all = (int64_t)a.T * a.q_heads;
            float *y = parts + (split * all + row) * D + 4 * hh;
#pragma unroll
            for (int j = 0; j < JT; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    *reinterpret_cast<float4 *>(y + 32 * j + 8 * k) =
                        make_float4(o[wr][j][4 * k], o[wr][j][4 * k + 1], o[wr][j][4 * k + 2], o[wr][j][4 * k + 3]);
            if (hh == 0) {
                float *s = parts + splits * all * D + (split * all + row) * 2;
                s[0] = m[wr];
                s[1] = l[wr];
            }
        }
    }
}

// Joins the splits of the rows that the tile kernel took, D / 4 threads a row.
template <int D, int DT>
__global__ __launch_bounds__(256) void kv_tile_join_kernel(const KvAttention a, int rows_min, int splits,
                                                           const float *parts) {
    constexpr int Q = D / 4;
    const int64_t all = (int64_t)a.T * a.q_heads;
    const int64_t row = (int64_t)blockIdx.x * (256 / Q) + threadIdx.x / Q;
    const int d4 = threadIdx.x % Q;
    if (row >= all) return;
    const int t = (int)(row / a.q_heads);
    if (a.cu_q && (t < a.cu_q[0] || t >= a.cu_q[a.B])) return;
    const KvSeq seq = kv_seq(a, a.cu_q ? kv_find(a.cu_q, a.B, t) : t);
    if ((int64_t)seq.nq * a.group < rows_min) return;
    const float *s = parts + splits * all * D;
    float mx = kNoMax;
    for (int i = 0; i < splits; ++i) mx = fmaxf(mx, s[(i * all + row) * 2]);
    float sum = 0.0f;
    f32x4 v = {0, 0, 0, 0};
    for (int i = 0; i < splits; ++i) {
        const float e = __builtin_amdgcn_exp2f(s[(i * all + row) * 2] - mx);
        sum += s[(i * all + row) * 2 + 1] * e;
        v += *reinterpret_cast<const f32x4 *>(parts + (i * all + row) * D + 4 * d4) * e;
    }
    const float inv = row_factor(sum, seq.over);
    reinterpret_cast<uint2 *>(a.y)[row * Q + d4] =
        make_uint2(pack16<DT>(v[0] * inv, v[1] * inv), pack16<DT>(v[2] * inv, v[3] * inv));
}

template <int D, int FMT, int DT, int WR>
static void launch_tile(const KvAttention &a, int rows_min, int splits, float *parts, hipStream_t stream) {
    const int64_t tiles = a.T * a.group / (128 * WR) + (a.B < a.T ? a.B : a.T);
    kv_tile_kernel<D, FMT, DT, WR><<<dim3((unsigned)(tiles * a.cache.heads), splits), 256, 0, stream>>>(a, rows_min, splits, parts);
    if (splits > 1) {
        const int64_t rows = a.T * a.q_heads, per = 256 / (D / 4);
        kv_tile_join_kernel<D, DT><<<(unsigned)((rows + per - 1) / per), 256, 0, stream>>>(a, rows_min, splits, parts);
    }
}

template <int D, int FMT, int DT>
static void launch_tile_wr(const KvAttention &a, int wr, int rows_min, int splits, float *parts, hipStream_t stream) {
    if constexpr (D < 256) {
        if (wr == 2) return launch_tile<D, FMT, DT, 2>(a, rows_min, splits, parts, stream);
    }
    launch_tile<D, FMT, DT, 1>(a, rows_min, splits, parts, stream);
}

template <int D>
static void launch_tile_d(const KvAttention &a, int dt, int wr, int rows_min, int splits, float *parts,
                          hipStream_t stream) {
    if (a.cache.fmt == E2M1) {
        if (dt == F16) launch_tile_wr<D, E2M1, F16>(a, wr, rows_min, splits, parts, stream);
        else launch_tile_wr<D, E2M1, BF16>(a, wr, rows_min, splits, parts, stream);
    } else {
        if (dt == F16) launch_tile_wr<D, E4M3, F16>(a, wr, rows_min, splits, parts, stream);
        else launch_tile_wr<D, E4M3, BF16>(a, wr, rows_min, splits, parts, stream);
    }
}

void launch_kv_tiles(const KvAttention &a, int dt, int wr, int rows_min, int splits, float *parts,
                     hipStream_t stream) {
    if (a.cache.dim == 64) launch_tile_d<64>(a, dt, wr, rows_min, splits, parts, stream);
    else if (a.cache.dim == 128) launch_tile_d<128>(a, dt, wr, rows_min, splits, parts, stream);
    else launch_tile_d<256>(a, dt, wr, rows_min, splits, parts, stream);
}

}  // namespace sq
