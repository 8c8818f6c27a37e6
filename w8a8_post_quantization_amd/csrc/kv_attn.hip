// Attention over the microscaled cache, few queries a sequence (include/sq_kv.h):
//   y = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  s_j = scale (q . k_j)
//
// The rows of an item - one sequence and key head, its queries times the query
// heads that share the key head - are the columns of the matrix instructions:
// S^T = K Q^T (16 keys x 16 rows, 32 channels an instruction) and
// O^T = V^T P^T (16 channels x 16 rows, 32 keys an instruction).  So laid out,
// a lane holds scores of one row in S^T just where the second product takes
// its weights, no lane exchanges data in the loop, and codes go from memory to
// the operands through registers alone: a lane's key operand is successive
// channels of one key (any order of the channels serves, the query's operand
// having the same), a value operand eight keys of one channel, whose pairs are
// joined by a byte permute after the conversion.
//
// Memory bound, so the work is cut into equal shares whatever the sequences'
// lengths: the tiles of 128 keys of all items in a row, a share of successive
// tiles a block.  An item inside a block's share is finished there; of an item
// across shares each block leaves its sum, maximum and weighted values in the
// workspace (at most two parts a block: the item it continues and the one it
// leaves off), and a second kernel joins them in the order of the blocks.
#include "kv_attn_device.h"

namespace sq {

constexpr int kTile = 128;       // keys of a unit of work: 32 for each of four waves
constexpr int kMaxBlocks = 1024;

// What a block leaves in the workspace for the joining kernel.
struct Part {
    int b, h, rows, last;  // the item that it begins and does not end; the block that ends it (-1: none)
};

template <int D, int NT> struct PartSize {
    static constexpr int rows = 16 * NT;
    static constexpr int floats = rows * (D + 2);  // values, maxima, sums
};

// 32 keys' codes and scales as a lane loads them.
template <int D, int FMT> struct Keys32 {
    static constexpr int NB = D / 32;
    static constexpr int KN = NB * (FMT == E2M1 ? 4 : 8);   // code bytes of a key, a quarter of its channels
    static constexpr int KS = NB < 4 ? 1 : NB / 4;          // scale bytes of those
    static constexpr int VN = FMT == E2M1 ? D / 32 : D / 16;  // code bytes of a value, a sixteenth of its channels
    Words<KN> k[2];
    uint32_t ks[2][KS];
    Words<VN> v[8];
    uint32_t vs[8];
};

template <int D, int FMT, int DT, int NT>
__global__ __launch_bounds__(256) void kv_attn_kernel(const KvAttention a, int rows_max) {
    constexpr int NB = D / 32, J = D / 16;  // blocks of a row; channel tiles
    using Raw = Keys32<D, FMT>;
    constexpr int RB = FMT == E2M1 ? D / 2 : D;  // code bytes of a row
    __shared__ int64_t s_pre[257];
    __shared__ int s_at[2];
    __shared__ float s_m[4][16 * NT], s_l[4][16 * NT];
    __shared__ f32x4 s_o[2][NT * J][64];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n16 = lane & 15, g = lane >> 4;
    const int heads = a.cache.heads, plog = a.cache.page_log, group = a.group;
    float *const work = reinterpret_cast<float *>(a.work);
    Part *const part = reinterpret_cast<Part *>(work);
    float *const parts = work + kMaxBlocks * sizeof(Part) / sizeof(float);

    const auto units_of = [&](const KvSeq &s) -> int {
        if (s.nq == 0 || (int64_t)s.nq * group > rows_max || s.hi <= s.lo) return 0;
        return (s.hi - (s.lo & ~15) + kTile - 1) / kTile;
    };
    // Units before each thread's stretch of sequences, and the whole sum.
    const int per_thread = (a.B + 255) / 256;
    const int b_first = tid * per_thread;
    {
        int64_t sum = 0;
        for (int i = 0; i < per_thread && b_first + i < a.B; ++i) sum += units_of(kv_seq(a, b_first + i));
        s_pre[tid + 1] = sum;
        if (tid == 0) s_pre[0] = 0;
        __syncthreads();
        for (int off = 1; off < 256; off <<= 1) {
            const int64_t v = tid >= off ? s_pre[tid + 1 - off] : 0;
            __syncthreads();
            s_pre[tid + 1] += v;
            __syncthreads();
        }
    }
    const int64_t total = s_pre[256] * heads;
    const int64_t share = (total + gridDim.x - 1) / gridDim.x;
    const int64_t u0 = share * blockIdx.x;
    const int64_t u1 = u0 + share < total ? u0 + share : total;
    if (tid == 0) part[blockIdx.x].last = -1;

    // The rows of a sequence with no units see no key.
    for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x) {
        const KvSeq s = kv_seq(a, (int)b);
        if (s.nq == 0 || (int64_t)s.nq * group > rows_max || units_of(s) != 0) continue;
        uint4 *y = reinterpret_cast<uint4 *>(a.y) + (int64_t)s.q0 * a.q_heads * (D / 8);
        const uint32_t w = s.over ? ~0u : 0u;
        for (int i = tid; i < s.nq * a.q_heads * (D / 8); i += 256) y[i] = make_uint4(w, w, w, w);
    }
    if (u0 >= u1) return;

    // The sequence that holds unit u0: the thread whose stretch has it walks it.
    if (s_pre[tid] * heads <= u0 && u0 < s_pre[tid + 1] * heads) {
        int64_t before = s_pre[tid] * heads;
        int b = b_first;
        for (;;) {
            const int64_t n = (int64_t)units_of(kv_seq(a, b)) * heads;
            if (u0 < before + n) break;
            before += n;
            ++b;
        }
        s_at[0] = b;
        s_at[1] = (int)(u0 - before);
    }
    __syncthreads();
    int b = __builtin_amdgcn_readfirstlane(s_at[0]);
    KvSeq seq = kv_seq(a, b);
    int units = units_of(seq);
    const int rem = __builtin_amdgcn_readfirstlane(s_at[1]);
    int h = __builtin_amdgcn_readfirstlane(rem / units);
    int tile = rem - h * units;

    const float c = a.scale * 1.44269504088896341f;
    for (int64_t u = u0; u < u1;) {
        const int count = (int)(u1 - u < units - tile ? u1 - u : units - tile);
        const int rows = seq.nq * group;
        const int first = seq.lo & ~15;
        const int ta = first + tile * kTile;
        const int te = ta + count * kTile < seq.hi ? ta + count * kTile : seq.hi;

        // The queries' operands, and the keys that each row sees.
        uint4 qf[NT][NB];
        int r_lo[NT], r_hi[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = nt * 16 + n16;
            const int i = r / group;
            const char *x = (const char *)a.q +
                            ((int64_t)(seq.q0 + i) * a.q_st + (int64_t)(h * group + r - i * group) * a.q_sh) * 2;
#pragma unroll
            for (int s = 0; s < NB; ++s) {
                qf[nt][s] = make_uint4(0, 0, 0, 0);
                if (r < rows) qf[nt][s] = reinterpret_cast<const uint4 *>(x)[g * NB + s];
            }
            const int p = seq.nk - seq.nq + i;
            r_hi[nt] = r < rows ? (a.causal ? p + 1 : seq.nk) : 0;
            r_lo[nt] = a.window && (int64_t)p - a.window + 1 > 0 ? (int)(p - a.window + 1) : 0;
        }
        // Every row sees the keys all_lo .. all_hi.
        const int all_hi = a.causal ? seq.nk - seq.nq + 1 : seq.nk;
        const int all_lo = a.window && (int64_t)seq.nk - a.window > 0 ? (int)(seq.nk - a.window) : 0;

        float m[NT], l[NT];
        f32x4 o[NT][J];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt] = kNoMax;
            l[nt] = 0.0f;
#pragma unroll
            for (int j = 0; j < J; ++j) o[nt][j] = f32x4{0, 0, 0, 0};
        }

        const int32_t *const table = a.table + (int64_t)b * a.width;
        const int g_last = (seq.hi - 1) >> 4;
        const auto load = [&](int t, Raw &r) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                int grp = (t >> 4) + half;
                grp = __builtin_amdgcn_readfirstlane(grp < g_last ? grp : g_last);
                int64_t page = table[grp >> (plog - 4)];
                const bool held = page >= 0 && page < a.cache.pages;
                page = held ? page : 0;
                const int64_t row = kv_row(a.cache, page, h, (grp & ((1 << (plog - 4)) - 1)) << 4);
                const uint8_t *kq = a.cache.kq + row * RB + n16 * RB + g * Raw::KN;
                r.k[half] = load_codes<Raw::KN>(kq);
                const uint8_t *ks = a.cache.ks + row * NB + n16 * NB + g * NB / 4;
#pragma unroll
                for (int i = 0; i < Raw::KS; ++i) r.ks[half][i] = held ? ks[i] : 255u;
                const uint8_t *vq = a.cache.vq + row * RB + 4 * g * RB + n16 * Raw::VN;
                const uint8_t *vs = a.cache.vs + row * NB + 4 * g * NB + n16 * NB / 16;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    r.v[4 * half + i] = load_codes<Raw::VN>(vq + i * RB);
                    r.vs[4 * half + i] = held ? vs[i * NB] : 255u;
                }
            }
        };
        const auto compute = [&](Raw &r, int t) {
            f32x4 st[NT][2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) st[nt][half] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < NB; ++s) {
                    const float sc = e8m0(r.ks[half][NB < 4 ? 0 : s / 4]);
                    const uint4 kf = codes8_to_16<FMT, DT>(&r.k[half].w[s * (FMT == E2M1 ? 1 : 2)], sc);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) st[nt][half] = mfma16<DT>(kf, qf[nt][s], st[nt][half]);
                }
            }
            const bool masked = t < all_lo || t + 32 > all_hi || t + 32 > te;
            if (masked) {
                // keys that no row sees (behind the last, before the window) are
                // taken as 0: what their place holds may be anything
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int key = t + 16 * (i >> 2) + 4 * g + (i & 3);
                    if (key < seq.lo || key >= te) {
                        r.vs[i] = 0;
                        r.v[i] = Words<Raw::VN>{};
                    }
                }
            }
            uint4 pf[NT], seen[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float x[8];
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = st[nt][i >> 2][i & 3] * c;
                if (masked) {
                    uint32_t v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int key = t + 16 * (i >> 2) + 4 * g + (i & 3);
                        const bool vis = key >= r_lo[nt] && key < r_hi[nt] && key < te;
                        x[i] = vis ? x[i] : -INFINITY;
                        v[i] = vis ? (DT == BF16 ? 0x3f80u : 0x3c00u) : 0u;
                    }
                    seen[nt] = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16,
                                          v[6] | v[7] << 16);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) top = fmaxf(top, x[i]);
                // The maximum may trail the true one by 8 (weights up to 256):
                // rows are rescaled only where it is passed by more.
                if (__any(top > m[nt] + 8.0f)) {
                    top = fmaxf(top, __shfl_xor(top, 16, 64));
                    top = fmaxf(top, __shfl_xor(top, 32, 64));
                    const float mn = fmaxf(m[nt], top);
                    const float f = __builtin_amdgcn_exp2f(m[nt] - mn);
                    m[nt] = mn;
                    l[nt] *= f;
#pragma unroll
                    for (int j = 0; j < J; ++j) o[nt][j] *= f;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[i] = __builtin_amdgcn_exp2f(x[i] - m[nt]);
                    l[nt] += x[i];
                }
                pf[nt] = make_uint4(pack16<DT>(x[0], x[1]), pack16<DT>(x[2], x[3]),
                                    pack16<DT>(x[4], x[5]), pack16<DT>(x[6], x[7]));
            }
            float sc[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) sc[i] = e8m0(r.vs[i]);
#pragma unroll
            for (int q = 0; q < J / 2; ++q) {
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = pair_of<FMT, DT>(r.v[i], q, sc[i]);
#pragma unroll
                for (int odd = 0; odd < 2; ++odd) {
                    const uint32_t sel = odd ? 0x07060302u : 0x05040100u;
                    uint4 vf = make_uint4(__builtin_amdgcn_perm(w[1], w[0], sel), __builtin_amdgcn_perm(w[3], w[2], sel),
                                          __builtin_amdgcn_perm(w[5], w[4], sel), __builtin_amdgcn_perm(w[7], w[6], sel));
                    const int j = 2 * q + odd;
                    if (masked && seq.nq > 1) {
                        // A weight of 0 does not keep an infinity or NaN from a
                        // row that must not see it: they are taken out, and
                        // brought to the rows that see them by a product of ones.
                        uint4 up, down;
                        vf.x = split_nonfinite<DT>(vf.x, up.x, down.x);
                        vf.y = split_nonfinite<DT>(vf.y, up.y, down.y);
                        vf.z = split_nonfinite<DT>(vf.z, up.z, down.z);
                        vf.w = split_nonfinite<DT>(vf.w, up.w, down.w);
                        const uint32_t any = up.x | up.y | up.z | up.w | down.x | down.y | down.z | down.w;
                        if (__any(any != 0)) {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                const f32x4 cu = mfma16<DT>(up, seen[nt], f32x4{0, 0, 0, 0});
                                const f32x4 cd = mfma16<DT>(down, seen[nt], f32x4{0, 0, 0, 0});
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    if (cu[i] > 0) o[nt][j][i] += INFINITY;
                                    if (cd[i] > 0) o[nt][j][i] -= INFINITY;
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) o[nt][j] = mfma16<DT>(vf, pf[nt], o[nt][j]);
                }
            }
        };
        {
            Raw r0, r1;
            int t = ta + 32 * wave;
            if (t < te) load(t, r0);
            while (t < te) {
                if (t + kTile < te) load(t + kTile, r1);
                compute(r0, t);
                t += kTile;
                if (t >= te) break;
                if (t + kTile < te) load(t + kTile, r0);
                compute(r1, t);
                t += kTile;
            }
        }

        // Join the waves: one maximum, then the values of waves 2 and 3 into 0
        // and 1, of 1 into 0.
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            l[nt] += __shfl_xor(l[nt], 16, 64);
            l[nt] += __shfl_xor(l[nt], 32, 64);
            if (g == 0) {
                s_m[wave][nt * 16 + n16] = m[nt];
                s_l[wave][nt * 16 + n16] = l[nt];
            }
        }
        __syncthreads();
        float mx[NT], sum[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = nt * 16 + n16;
            mx[nt] = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
            sum[nt] = 0.0f;
#pragma unroll
            for (int w = 0; w < 4; ++w) sum[nt] += s_l[w][r] * __builtin_amdgcn_exp2f(s_m[w][r] - mx[nt]);
            const float f = __builtin_amdgcn_exp2f(m[nt] - mx[nt]);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                o[nt][j] *= f;
                if (wave >= 2) s_o[wave - 2][nt * J + j][lane] = o[nt][j];
            }
        }
        __syncthreads();
        if (wave < 2) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    o[nt][j] += s_o[wave][nt * J + j][lane];
                    if (wave == 1) s_o[1][nt * J + j][lane] = o[nt][j];
                }
        }
        __syncthreads();
        const bool whole = count == units;
        if (wave == 0) {
            // a lane's values are D / 4 successive channels of its row
            const int slot = tile > 0 ? 0 : 1;
            float *const out = parts + (int64_t)(blockIdx.x * 2 + slot) * PartSize<D, NT>::floats;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int r = nt * 16 + n16;
                float v[D / 4];
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const f32x4 x = o[nt][j] + s_o[1][nt * J + j][lane];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i * J + j] = x[i];
                }
                if (r < rows) {
                    if (whole) {
                        const float inv = row_factor(sum[nt], seq.over);
                        const int i = r / group;
                        uint4 *y = reinterpret_cast<uint4 *>(a.y) +
                                   (((int64_t)(seq.q0 + i) * a.q_heads + h * group + r - i * group) * D + g * (D / 4)) / 8;
#pragma unroll
                        for (int k = 0; k < D / 32; ++k)
                            y[k] = make_uint4(pack16<DT>(v[8 * k] * inv, v[8 * k + 1] * inv),
                                              pack16<DT>(v[8 * k + 2] * inv, v[8 * k + 3] * inv),
                                              pack16<DT>(v[8 * k + 4] * inv, v[8 * k + 5] * inv),
                                              pack16<DT>(v[8 * k + 6] * inv, v[8 * k + 7] * inv));
                    } else {
                        float4 *y = reinterpret_cast<float4 *>(out + r * D + g * (D / 4));
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            y[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                        if (g == 0) {
                            out[16 * NT * D + r] = mx[nt];
                            out[16 * NT * D + 16 * NT + r] = sum[nt];
                        }
                    }
                }
            }
            if (lane == 0 && !whole && tile == 0) {
                Part p;
                p.b = b;
                p.h = h;
                p.rows = rows;
                p.last = (int)((u + units - 1) / share);
                part[blockIdx.x] = p;
            }
        }
        u += count;
        if (u >= u1) break;
        __syncthreads();  // (s_m, s_l and s_o are written again)
        tile = 0;
        if (++h == heads) {
            h = 0;
            do {
                seq = kv_seq(a, ++b);
                units = units_of(seq);
            } while (units == 0);
        }
    }
}

// Joins the parts of the item that block blockIdx.x began and did not end, one
// row a block: 256 threads are D / 4 channel quads by as many of the parts at a
// time.
template <int D, int DT, int NT>
__global__ __launch_bounds__(256) void kv_join_kernel(const KvAttention a) {
    constexpr int Q = D / 4, W = 256 / Q;
    const float *const work = reinterpret_cast<const float *>(a.work);
    const Part p = reinterpret_cast<const Part *>(work)[blockIdx.x];
    const int r = blockIdx.y;
    if (p.last < 0 || r >= p.rows) return;
    const float *const parts = work + kMaxBlocks * sizeof(Part) / sizeof(float);
    __shared__ f32x4 s_o[W][Q];
    __shared__ float s_m[W], s_l[W];
    const int d4 = threadIdx.x % Q, w = threadIdx.x / Q;
    const int first = blockIdx.x, n = p.last - first + 1;
    float m = kNoMax, l = 0.0f;
    f32x4 o = {0, 0, 0, 0};
    for (int i = w; i < n; i += W) {
        // (the first block's part is its second: it begins the item)
        const float *x = parts + (int64_t)((first + i) * 2 + (i == 0)) * PartSize<D, NT>::floats;
        const float pm = x[16 * NT * D + r], pl = x[16 * NT * D + 16 * NT + r];
        const f32x4 v = *reinterpret_cast<const f32x4 *>(x + r * D + 4 * d4);
        const float mn = fmaxf(m, pm);
        const float f = __builtin_amdgcn_exp2f(m - mn), e = __builtin_amdgcn_exp2f(pm - mn);
        l = l * f + pl * e;
        o = o * f + v * e;
        m = mn;
    }
    s_o[w][d4] = o;
    if (d4 == 0) {
        s_m[w] = m;
        s_l[w] = l;
    }
    __syncthreads();
    if (w != 0) return;
    float mx = s_m[0];
    for (int i = 1; i < W; ++i) mx = fmaxf(mx, s_m[i]);
    float sum = 0.0f;
    f32x4 v = {0, 0, 0, 0};
    for (int i = 0; i < W; ++i) {
        const float e = __builtin_amdgcn_exp2f(s_m[i] - mx);
        sum += s_l[i] * e;
        v += s_o[i][d4] * e;
    }
    const KvSeq seq = kv_seq(a, p.b);
    const float inv = row_factor(sum, seq.over);
    const int i = r / a.group;
    uint2 *y = reinterpret_cast<uint2 *>(a.y) +
               (((int64_t)(seq.q0 + i) * a.q_heads + p.h * a.group + r - i * a.group) * D + 4 * d4) / 4;
    *y = make_uint2(pack16<DT>(v[0] * inv, v[1] * inv), pack16<DT>(v[2] * inv, v[3] * inv));
}

// Which kernels a call takes.
struct Plan {
    int nt;             // column groups of 16 rows of the kernel above; 0: not used
    int rows_max;       // it takes the sequences of up to so many rows
    int64_t blocks;
    int wr;             // row groups a wave of the tile kernel; 0: not used
    int splits;
    size_t tile_parts;  // where its parts begin in the workspace
    size_t bytes;
};

static Plan plan_attention(int64_t T, int q_heads, int heads, int dim, int B, int64_t keys, int64_t max_q) {
    Plan p = {};
    const int64_t group = q_heads / heads, most = max_q * group;
    // Up to 32 rows the first kernel has all. Of a call with longer sequences it
    // takes those of up to 16 rows (or of one query), the tile kernel the others.
    p.nt = most <= 16 ? 1 : most <= 32 ? 2 : group <= 16 ? 1 : group <= 32 ? 2 : 0;
    p.rows_max = (int)(most < 16 * p.nt ? most : 16 * p.nt);
    if (p.nt) {
        const int64_t units = (int64_t)B * heads * ((keys + 15 + kTile - 1) / kTile);
        p.blocks = units < kMaxBlocks ? (units > 0 ? units : 1) : kMaxBlocks;
        p.bytes = kMaxBlocks * sizeof(Part) + (size_t)p.blocks * 2 * 16 * p.nt * (dim + 2) * sizeof(float);
    }
    if (most > 32) {
        p.wr = dim == 256 || most <= 128 ? 1 : 2;
        const int64_t tiles = (T * group + 128 * p.wr - 1) / (128 * p.wr) * heads;
        // few tiles: the keys of each are split over blocks
        int64_t splits = tiles >= 256 ? 1 : 512 / tiles;
        if (splits > (keys + 511) / 512) splits = (keys + 511) / 512;
        p.splits = (int)(splits > 16 ? 16 : splits < 1 ? 1 : splits);
        p.tile_parts = (p.bytes + 255) & ~(size_t)255;
        if (p.splits > 1) p.bytes = p.tile_parts + (size_t)p.splits * T * q_heads * (dim + 2) * sizeof(float);
    }
    return p;
}

size_t kv_attention_workspace(int64_t T, int q_heads, int heads, int dim, int B, int64_t keys, int64_t max_q) {
    return plan_attention(T, q_heads, heads, dim, B, keys, max_q).bytes;
}

template <int D, int FMT, int DT, int NT>
static void launch_attn(const KvAttention &a, const Plan &p, hipStream_t stream) {
    kv_attn_kernel<D, FMT, DT, NT><<<(unsigned)p.blocks, 256, 0, stream>>>(a, p.rows_max);
    if (p.blocks > 1)
        kv_join_kernel<D, DT, NT><<<dim3((unsigned)p.blocks, p.rows_max), 256, 0, stream>>>(a);
}

template <int D, int FMT, int DT>
static void launch_attn_nt(const KvAttention &a, const Plan &p, hipStream_t stream) {
    if (p.nt == 1) launch_attn<D, FMT, DT, 1>(a, p, stream);
    else launch_attn<D, FMT, DT, 2>(a, p, stream);
}

template <int D>
static void launch_attn_d(const KvAttention &a, const Plan &p, int dt, hipStream_t stream) {
    if (a.cache.fmt == E2M1) {
        if (dt == F16) launch_attn_nt<D, E2M1, F16>(a, p, stream);
        else launch_attn_nt<D, E2M1, BF16>(a, p, stream);
    } else {
        if (dt == F16) launch_attn_nt<D, E4M3, F16>(a, p, stream);
        else launch_attn_nt<D, E4M3, BF16>(a, p, stream);
    }
}

void launch_kv_attention(const KvAttention &a, int64_t max_q, int dt, hipStream_t stream) {
    const Plan p = plan_attention(a.T, a.q_heads, a.cache.heads, a.cache.dim, a.B,
                                  a.width << a.cache.page_log, max_q);
    if (p.nt) {
        if (a.cache.dim == 64) launch_attn_d<64>(a, p, dt, stream);
        else if (a.cache.dim == 128) launch_attn_d<128>(a, p, dt, stream);
        else launch_attn_d<256>(a, p, dt, stream);
    }
    if (p.wr)
        launch_kv_tiles(a, dt, p.wr, p.rows_max + 1, p.splits,
                        reinterpret_cast<float *>((char *)a.work + p.tile_parts), stream);
}

}  // namespace sq
