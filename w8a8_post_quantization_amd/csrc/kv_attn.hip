// Attention over the microscaled cache, few queries a sequence (include/sq_kv.h):
//   y = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  s_j = scale (q . k_j)
//
// The rows of an item - one sequence and key head, its queries times the query
// heads that share the key head - are the columns of the matrix instructions:
// S^T = K Q^T (16 keys x 16 rows, 32 channels an instruction) and
// O^T = V^T P^T (16 channels x 16 rows, 32 keys an instruction).  So laid out,
// a lane holds scores of one row in S^T just where the second product takes
// its weights, and no lane exchanges data in the loop.  Codes go from memory to
// a ring of tiles in LDS, each wave's its own, by loads that take no registers,
// and are converted as they are read from there: a lane's key operand is
// successive channels of one key (any order of the channels serves, the query's
// operand having the same), a value operand eight keys of one channel, whose
// pairs are joined by a byte permute after the conversion.
//
// Memory bound, so the work is cut into equal shares whatever the sequences'
// lengths: the tiles of 128 keys of all items in a row, a share of successive
// tiles a block.  An item inside a block's share is finished there; of an item
// across shares each block leaves its sum, maximum and weighted values in the
// workspace (at most two parts a block: the item it continues and the one it
// leaves off), and a second kernel joins them in the order of the blocks.
//
// 64 tokens over 130 .. 32768 keys, 64 / 8 heads of 128, e2m1: 86 us, 425 MB at
// 4.9 TB/s (without the arithmetic, in a copy for timing, 74); with codes loaded
// to registers it was 147.  A wave issues 253 vector, 108 scalar and 23 LDS
// instructions for 32 keys, which fill 59 % of the vector units' cycles.  16
// tokens over 900 .. 2300 keys, 56 heads of 128, e4m3: 64 us, 5.6 TB/s.  One
// token over 2049 keys, 64 / 8 heads: 7.7 us and 3.9 of the joining kernel.
#include "kv_attn_device.h"

namespace sq {

constexpr int kTile = 128;       // keys of a unit of work: 32 for each of four waves
constexpr int kMaxBlocks = 1024;  // (at most, whatever a CU holds)

// What a block leaves in the workspace for the joining kernel.
struct Part {
    int b, h, rows, last;  // the item that it begins and does not end; the block that ends it (-1: none)
};

template <int D, int NT> struct PartSize {
    static constexpr int rows = 16 * NT;
    static constexpr int floats = rows * (D + 2);  // values, maxima, sums
};

// 32 keys' codes and scales in a wave's LDS ring: the keys' codes, the values',
// then the keys' scales and the values', as they lie in the cache.
template <int D, int FMT> struct Tile32 {
    static constexpr int NB = D / 32;
    static constexpr int RB = FMT == E2M1 ? D / 2 : D;        // code bytes of a row
    static constexpr int KN = RB / 4;                         // of those, a lane's of a key: a quarter
    static constexpr int KS = NB < 4 ? 1 : NB / 4;            // scale bytes of a quarter
    static constexpr int VN = RB / 16;                        // a lane's of a value: a sixteenth
    static constexpr int codes = 32 * RB, scales = 32 * NB;
    static constexpr int scale_loads = 2 * scales > 256 ? 2 * scales / 256 : 1;
    static constexpr int loads = 2 * codes / 1024 + scale_loads;
    static constexpr int bytes = 2 * codes + 256 * scale_loads;
    // As many tiles in flight as a CU's LDS has room for with 3 blocks (2 where
    // a tile is 8 KB, 1 where it is 17 KB).
    static constexpr int stages = bytes < 4096 ? 4 : bytes < 8192 ? 3 : 2;
};
constexpr int kCus = 256;
// Blocks of the kernel on a CU: LDS allows 3, 2 or 1 of them, registers 2 with
// two column groups.
constexpr int blocks_per_cu(int dim, int fmt, int nt) {
    const int row = fmt == E2M1 ? dim / 2 : dim;  // code bytes: 32 to 256
    const int n = row <= 64 ? 3 : row <= 128 ? 2 : 1;
    return nt == 1 || n < 2 ? n : 2;
}

template <int D, int FMT, int DT, int NT>
__global__ __launch_bounds__(256, (blocks_per_cu(D, FMT, NT))) void kv_attn_kernel(
    const KvAttention a, int rows_max, const int32_t *__restrict__ tables) {
    using L = Tile32<D, FMT>;
    constexpr int NB = L::NB, RB = L::RB, J = D / 16;  // blocks, code bytes of a row; channel tiles
    constexpr int kRing = 4 * L::stages * L::bytes, kJoin = 4 * NT * J * 64 * 16;
    __shared__ int s_at[2];
    __shared__ KvSeq s_seq;
    __shared__ float s_m[4][16 * NT], s_l[4][16 * NT];
    // first the sequences' units, then the waves' rings, and (an item's keys
    // read) the join of the waves' sums
    __shared__ __attribute__((aligned(1024))) uint8_t s_ring[kRing > kJoin ? kRing : kJoin];
    int64_t *const s_pre = reinterpret_cast<int64_t *>(s_ring), *const s_wave = s_pre + 257;
    const auto s_o = reinterpret_cast<float(*)[64]>(s_ring);

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n16 = lane & 15, g = lane >> 4;
    const int heads = a.cache.heads, plog = a.cache.page_log, group = a.group;
    float *const work = reinterpret_cast<float *>(a.work);
    Part *const part = reinterpret_cast<Part *>(work);
    float *const parts = work + kMaxBlocks * sizeof(Part) / sizeof(float);

    const auto units_of = [&](const KvSeq &s) SQ_INLINE -> int {
        if (s.nq == 0 || (int64_t)s.nq * group > rows_max || s.hi <= s.lo) return 0;
        return (s.hi - (s.lo & ~15) + kTile - 1) / kTile;
    };
    // Units before each thread's stretch of sequences, and the whole sum.
    const int per_thread = (a.B + 255) / 256;
    const int b_first = tid * per_thread;
    {
        int64_t sum = 0;
        for (int i = 0; i < per_thread && b_first + i < a.B; ++i) sum += units_of(kv_seq(a, b_first + i));
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int64_t v = __shfl_up(sum, off, 64);
            if (lane >= off) sum += v;
        }
        if (lane == 63) s_wave[wave] = sum;
        __syncthreads();
        for (int w = 0; w < wave; ++w) sum += s_wave[w];
        s_pre[tid + 1] = sum;
        if (tid == 0) s_pre[0] = 0;
        __syncthreads();
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
        KvSeq s = kv_seq(a, b);
        for (;;) {
            const int64_t n = (int64_t)units_of(s) * heads;
            if (u0 < before + n) break;
            before += n;
            s = kv_seq(a, ++b);
        }
        s_at[0] = b;
        s_at[1] = (int)(u0 - before);
        s_seq = s;
    }
    __syncthreads();
    int b = __builtin_amdgcn_readfirstlane(s_at[0]);
    KvSeq seq = s_seq;
    int units = units_of(seq);
    const int rem = __builtin_amdgcn_readfirstlane(s_at[1]);
    int h = __builtin_amdgcn_readfirstlane(rem / units);
    int tile = rem - h * units;

    const float c = a.scale * 1.44269504088896341f;
    uint8_t *const ring = s_ring + wave * L::stages * L::bytes;
    const uint32_t ring_at = (uint32_t)(uintptr_t)(lds_void_t *)ring;
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

        const int32_t *const table = tables + (int64_t)b * a.width;
        const int g_last = (seq.hi - 1) >> 4;
        // A tile's loads go to LDS by themselves, so that tiles in flight take no
        // registers.  Its pages are looked up a tile ahead; whether each was in
        // the cache is kept as two bits a tile, the newest lowest.
        int page[2];
        uint32_t missing = 0;
        const auto look_up = [&](int t) SQ_INLINE {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int grp = (t >> 4) + half;
                page[half] = table[__builtin_amdgcn_readfirstlane(grp < g_last ? grp : g_last) >> (plog - 4)];
            }
        };
        const auto load = [&](int t, int slot) SQ_INLINE {
            int64_t row[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int grp = (t >> 4) + half;
                const int in_page = __builtin_amdgcn_readfirstlane((grp < g_last ? grp : g_last) & ((1 << (plog - 4)) - 1));
                const int p = __builtin_amdgcn_readfirstlane(page[half]);
                const bool held = p >= 0 && p < a.cache.pages;
                missing = missing << 1 | (held ? 0 : 1);
                row[half] = kv_row(a.cache, held ? p : 0, h, in_page << 4);
            }
            look_up(t + kTile);
            const int8_t *from[2 * L::codes / 1024];
#pragma unroll
            for (int i = 0; i < 2 * L::codes / 1024; ++i) {
                const uint8_t *q = i < L::codes / 1024 ? a.cache.kq : a.cache.vq;
                const int at = i * 1024 % L::codes;
                if constexpr (16 * RB >= 1024) {
                    from[i] = (const int8_t *)(q + row[at / (16 * RB)] * RB) + (uint32_t)(at % (16 * RB) + lane * 16);
                } else {  // (both groups of 16 keys in one load)
                    from[i] = (const int8_t *)(q + (lane < 32 ? row[0] : row[1]) * RB) + (uint32_t)(lane % 32 * 16);
                }
            }
            const uint32_t to = ring_at + slot * L::bytes;
            lds_dma_run<2 * L::codes / 1024, true>(from, to);
#pragma unroll
            for (int i = 0; i < L::scale_loads; ++i) {
                constexpr int W = L::scales / 4;  // words of 32 keys' scales
                const int w = (i * 64 + lane) % (2 * W);
                const uint8_t *e = w < W ? a.cache.ks : a.cache.vs;
                lds_dma4(e + (w % W < W / 2 ? row[0] : row[1]) * NB + w % (W / 2) * 4, to + 2 * L::codes + i * 256);
            }
        };
        const auto compute = [&](int t, int slot, uint32_t gone) SQ_INLINE {
            const bool masked = t < all_lo || t + 32 > all_hi || t + 32 > te;
            const uint8_t *const kq = ring + slot * L::bytes, *const vq = kq + L::codes;
            const uint8_t *const ks = vq + L::codes, *const vs = ks + L::scales;
            Words<L::KN> k[2];
            uint32_t ke[2][L::KS];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                k[half] = load_codes<L::KN>(kq + (16 * half + n16) * RB + g * L::KN);
#pragma unroll
                for (int i = 0; i < L::KS; ++i) ke[half][i] = ks[(16 * half + n16) * NB + g * NB / 4 + i];
            }
            Words<L::VN> v[8];
            uint32_t ve[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int key = 16 * (i >> 2) + 4 * g + (i & 3);
                v[i] = load_codes<L::VN>(vq + key * RB + n16 * L::VN);
                ve[i] = vs[key * NB + n16 * NB / 16];
            }
            if (gone) {  // pages that are not in the cache: NaN
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t nan = gone >> (1 - half) & 1 ? 255u : 0u;
#pragma unroll
                    for (int i = 0; i < L::KS; ++i) ke[half][i] |= nan;
#pragma unroll
                    for (int i = 0; i < 4; ++i) ve[4 * half + i] |= nan;
                }
            }
            f32x4 st[NT][2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) st[nt][half] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < NB; ++s) {
                    const float sc = e8m0(ke[half][NB < 4 ? 0 : s / 4]);
                    const uint4 kf = codes8_to_16<FMT, DT>(&k[half].w[s * (FMT == E2M1 ? 1 : 2)], sc);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) st[nt][half] = mfma16<DT>(kf, qf[nt][s], st[nt][half]);
                }
            }
            uint32_t apart = 0;
            if (masked) {
                asm volatile("");  // (a branch, not selects)
                // keys that no row sees (behind the last, before the window) are
                // taken as 0: what their place holds may be anything
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int key = t + 16 * (i >> 2) + 4 * g + (i & 3);
                    const bool none = key < seq.lo || key >= te;
                    // A weight of 0 does not keep an infinity or NaN from a row
                    // that must not see it: such keys are taken on their own.
                    const bool alone = !none && seq.nq > 1 && may_be_nonfinite<FMT, DT>(v[i], ve[i]);
                    const uint64_t who = __ballot(alone);
                    // (a key is the lanes of one g; the whole key is set apart)
                    const bool mine = (who >> (16 * g) & 0xffff) != 0;
#pragma unroll
                    for (int n = 0; n < 4; ++n)
                        if (who >> (16 * n) & 0xffff) apart |= 1u << (16 * (i >> 2) + 4 * n + (i & 3));
                    if (none || mine) {
                        ve[i] = 0;
                        v[i] = Words<L::VN>{};
                    }
                }
            }
            apart = __builtin_amdgcn_readfirstlane(apart);
            uint4 pf[NT];
            float x[NT][8];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < 8; ++i) x[nt][i] = st[nt][i >> 2][i & 3] * c;
                if (masked) {
                    asm volatile("");
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int key = t + 16 * (i >> 2) + 4 * g + (i & 3);
                        if (key < r_lo[nt] || key >= r_hi[nt] || key >= te) x[nt][i] = -INFINITY;
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) top = fmaxf(top, x[nt][i]);
                // Rows are rescaled only where the maximum trails by more than it may.
                if (__any(top - m[nt] > kTrail + kLift<DT>)) {
                    top = fmaxf(top, __shfl_xor(top, 16, 64));
                    top = fmaxf(top, __shfl_xor(top, 32, 64));
                    const float mn = fmaxf(m[nt], top - kLift<DT>);
                    const float f = __builtin_amdgcn_exp2f(m[nt] - mn);
                    m[nt] = mn;
                    l[nt] *= f;
#pragma unroll
                    for (int j = 0; j < J; ++j) o[nt][j] *= f;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[nt][i] = __builtin_amdgcn_exp2f(x[nt][i] - m[nt]);
                    l[nt] += x[nt][i];
                }
                pf[nt] = make_uint4(pack16<DT>(x[nt][0], x[nt][1]), pack16<DT>(x[nt][2], x[nt][3]),
                                    pack16<DT>(x[nt][4], x[nt][5]), pack16<DT>(x[nt][6], x[nt][7]));
            }
            float sc[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) sc[i] = e8m0(ve[i]);
#pragma unroll
            for (int q = 0; q < J / 2; ++q) {
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = pair_of<FMT, DT>(v[i], q, sc[i]);
#pragma unroll
                for (int odd = 0; odd < 2; ++odd) {
                    const uint32_t sel = odd ? 0x07060302u : 0x05040100u;
                    const uint4 vf = make_uint4(__builtin_amdgcn_perm(w[1], w[0], sel), __builtin_amdgcn_perm(w[3], w[2], sel),
                                          __builtin_amdgcn_perm(w[5], w[4], sel), __builtin_amdgcn_perm(w[7], w[6], sel));
                    const int j = 2 * q + odd;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) o[nt][j] = mfma16<DT>(vf, pf[nt], o[nt][j]);
                }
            }
            // (rare) The keys set apart, one at a time, for the rows that see them.
            for (; apart; apart &= apart - 1) {
                const int n = __builtin_ctz(apart), i = 4 * (n >> 4) + (n & 3), from = n16 + 16 * ((n >> 2) & 3);
                const int key = t + n;
                const uint32_t nan = gone >> (1 - (n >> 4)) & 1 ? 255u : 0u;
                float w[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float p = x[nt][0];
#pragma unroll
                    for (int z = 1; z < 8; ++z) p = z == i ? x[nt][z] : p;
                    w[nt] = __shfl(p, from, 64);
                }
#pragma unroll
                for (int z = 0; z < 4; ++z) {  // J channels from J (4 g + z) on
                    const Words<L::VN> c = load_codes<L::VN>(vq + n * RB + (4 * g + z) * L::VN);
                    const uint32_t e = vs[n * NB + (4 * g + z) * NB / 16] | nan;
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        const float val = half_of<DT>(pair_of<FMT, DT>(c, j >> 1, e8m0(e)), j & 1);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            if (key >= r_lo[nt] && key < r_hi[nt]) o[nt][j][z] += w[nt] * val;
                    }
                }
            }
        };
        const int t0 = ta + 32 * wave;
        const int n_tiles = t0 < te ? (te - t0 + kTile - 1) / kTile : 0;
        if (n_tiles) {
            look_up(t0);
            int slot = 0;  // of the next load
            for (int i = 0; i < L::stages - 1 && i < n_tiles; ++i) load(t0 + i * kTile, slot++);
            int read = 0;
            for (int i = 0; i < n_tiles; ++i) {
                const int more = n_tiles - 1 - i;
                if (more >= L::stages - 1) {
                    // (the slot's last reads have returned)
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    load(t0 + (i + L::stages - 1) * kTile, slot);
                    slot = slot + 1 == L::stages ? 0 : slot + 1;
                }
                const int later = more < L::stages - 1 ? more : L::stages - 1;
                wait_stages<L::stages - 1, L::loads>(later);
                asm volatile("" ::: "memory");
                compute(t0 + i * kTile, read, missing >> (2 * later) & 3);
                read = read + 1 == L::stages ? 0 : read + 1;
            }
        }

        // Join the waves: one maximum; the values through LDS, a quarter of the
        // channels a wave.  (All loads to the rings have been waited for.)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            l[nt] += __shfl_xor(l[nt], 16, 64);
            l[nt] += __shfl_xor(l[nt], 32, 64);
            if (g == 0) {
                s_m[wave][nt * 16 + n16] = m[nt];
                s_l[wave][nt * 16 + n16] = l[nt];
            }
        }
        __syncthreads();  // (the rings are read, too)
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
                const f32x4 v = o[nt][j] * f;
#pragma unroll
                for (int i = 0; i < 4; ++i) s_o[((wave * 4 + i) * NT + nt) * J + j][lane] = v[i];
            }
        }
        __syncthreads();
        const bool whole = count == units;
        {
            // value `wave` of a lane's four: J successive channels of its row
            const int slot = tile > 0 ? 0 : 1;
            float *const out = parts + (int64_t)(blockIdx.x * 2 + slot) * PartSize<D, NT>::floats;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int r = nt * 16 + n16;
                float v[J];
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    v[j] = 0.0f;
#pragma unroll
                    for (int w = 0; w < 4; ++w) v[j] += s_o[((w * 4 + wave) * NT + nt) * J + j][lane];
                }
                if (r < rows) {
                    const int d = J * (4 * g + wave);
                    if (whole) {
                        const int i = r / group;
                        const float inv = row_factor(sum[nt], r_hi[nt], seq.over);
                        uint2 *y = reinterpret_cast<uint2 *>(a.y) +
                                   (((int64_t)(seq.q0 + i) * a.q_heads + h * group + r - i * group) * D + d) / 4;
#pragma unroll
                        for (int k = 0; k < J / 4; ++k)
                            y[k] = make_uint2(pack16<DT>(v[4 * k] * inv, v[4 * k + 1] * inv),
                                              pack16<DT>(v[4 * k + 2] * inv, v[4 * k + 3] * inv));
                    } else {
                        float4 *y = reinterpret_cast<float4 *>(out + r * D + d);
#pragma unroll
                        for (int k = 0; k < J / 4; ++k)
                            y[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                        if (g == 0 && wave == 0) {
                            out[16 * NT * D + r] = mx[nt];
                            out[16 * NT * D + 16 * NT + r] = sum[nt];
                        }
                    }
                }
            }
            if (tid == 0 && !whole && tile == 0) {
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

// Joins the parts of the item that block blockIdx.x began and did not end, a
// row a time: 256 threads are D / 4 channel quads by W of the parts at a time.
// All that a row's first W kAhead parts hold is asked for at once, before the
// maximum is known: the kernel is a chain of memory latencies.
template <int D, int DT, int NT>
__global__ __launch_bounds__(256) void kv_join_kernel(const KvAttention a) {
    constexpr int Q = D / 4, W = 256 / Q, kAhead = 4, kRows = 16 * NT;
    const float *const work = reinterpret_cast<const float *>(a.work);
    const Part p = reinterpret_cast<const Part *>(work)[blockIdx.x];
    if (p.last < 0) return;
    const float *const parts = work + kMaxBlocks * sizeof(Part) / sizeof(float);
    __shared__ f32x4 s_o[W][Q];
    __shared__ float s_f[kMaxBlocks], s_red[4];
    const int tid = threadIdx.x, d4 = tid % Q, w = tid / Q;
    const int first = blockIdx.x, n = p.last - first + 1;
    const KvSeq seq = kv_seq(a, p.b);
    // (the first block's part is its second: it begins the item)
    const auto part = [&](int i) SQ_INLINE {
        return parts + (int64_t)((first + i) * 2 + (i == 0)) * PartSize<D, NT>::floats;
    };
    const auto reduced = [&](float v, auto op) SQ_INLINE {
#pragma unroll
        for (int off = 32; off; off >>= 1) v = op(v, __shfl_xor(v, off, 64));
        if ((tid & 63) == 0) s_red[tid >> 6] = v;
        __syncthreads();
        v = op(op(s_red[0], s_red[1]), op(s_red[2], s_red[3]));
        __syncthreads();
        return v;
    };
    for (int r = blockIdx.y; r < p.rows; r += gridDim.y) {
        f32x4 ahead[kAhead];
#pragma unroll
        for (int z = 0; z < kAhead; ++z) {
            const int i = w + z * W;
            ahead[z] = *reinterpret_cast<const f32x4 *>(part(i < n ? i : n - 1) + r * D + 4 * d4);
        }
        float mx = kNoMax, sum = 0.0f;
        for (int i = tid; i < n; i += 256) {
            s_f[i] = part(i)[kRows * D + r];
            mx = fmaxf(mx, s_f[i]);
        }
        float l = tid < n ? part(tid)[kRows * D + kRows + r] : 0.0f;
        mx = reduced(mx, [](float x, float y) { return fmaxf(x, y); });
        for (int i = tid; i < n; i += 256) {
            s_f[i] = __builtin_amdgcn_exp2f(s_f[i] - mx);
            if (i >= 256) l = part(i)[kRows * D + kRows + r];
            sum += l * s_f[i];
        }
        sum = reduced(sum, [](float x, float y) { return x + y; });
        f32x4 o = {0, 0, 0, 0};
#pragma unroll
        for (int z = 0; z < kAhead; ++z)
            if (w + z * W < n) o += ahead[z] * s_f[w + z * W];
#pragma unroll 4
        for (int i = w + kAhead * W; i < n; i += W)
            o += *reinterpret_cast<const f32x4 *>(part(i) + r * D + 4 * d4) * s_f[i];
        s_o[w][d4] = o;
        __syncthreads();
        if (w == 0) {
            f32x4 v = o;
            for (int i = 1; i < W; ++i) v += s_o[i][d4];
            const int i = r / a.group;
            const float inv = row_factor(sum, keys_end(a, seq, i), seq.over);
            uint2 *y = reinterpret_cast<uint2 *>(a.y) +
                       (((int64_t)(seq.q0 + i) * a.q_heads + p.h * a.group + r - i * a.group) * D + 4 * d4) / 4;
            *y = make_uint2(pack16<DT>(v[0] * inv, v[1] * inv), pack16<DT>(v[2] * inv, v[3] * inv));
        }
        // (s_o and s_f are written again behind two barriers)
    }
}

// Which kernels a call takes.
struct Plan {
    int nt;             // column groups of 16 rows of the kernel above; 0: not used
    int rows_max;       // it takes the sequences of up to so many rows
    int64_t blocks;
    int waves;          // of a block of the tile kernel, 32 rows each; 0: not used
    int splits;
    size_t tile_parts;  // where its parts begin in the workspace
    size_t bytes;
};

static Plan plan_attention(int64_t T, int q_heads, int heads, int dim, int fmt, int B, int64_t keys,
                           int64_t max_q) {
    Plan p = {};
    const int64_t group = q_heads / heads, most = max_q * group;
    // Up to 32 rows (16 with 256 channels: registers) the first kernel has all:
    // 24 rows over 4000 .. 8000 keys, 16 sequences of 4 heads of 128, take it
    // 26 us, and the tile kernel 50 + 11 with 128 channels, 20 against 39 + 11
    // with 64.  Of a call with longer sequences it takes those of up to 16 rows
    // (or of one query), the tile kernel the others.
    const int two = dim == 256 ? 0 : 2;
    p.nt = most <= 16 ? 1 : most <= 32 && two ? two : group <= 16 ? 1 : group <= 32 ? two : 0;
    p.rows_max = (int)(most < 16 * p.nt ? most : 16 * p.nt);
    if (p.nt) {
        const int64_t units = (int64_t)B * heads * ((keys + 15 + kTile - 1) / kTile);
        const int64_t most_blocks = (int64_t)kCus * blocks_per_cu(dim, fmt, p.nt);
        p.blocks = units < most_blocks ? (units > 0 ? units : 1) : most_blocks;
        p.bytes = kMaxBlocks * sizeof(Part) + (size_t)p.blocks * 2 * 16 * p.nt * (dim + 2) * sizeof(float);
    }
    if (most > 16 * p.nt) {
        // With 128 channels eight waves share what a block converts where they
        // have rows (a prompt of 8192, 64 / 8 heads: 1251 us, with four 1372; 256
        // rows over 2000 .. 8000 keys: 76 and 78); up to 128 rows four waves do
        // (128 rows: 46 us, with eight 71; 64 rows over 4000 keys: 27 and 31).
        // With 64 channels four waves, three blocks a CU (windowed chunks of 77 ..
        // 1013: 53 us, with eight 67; a prompt of 8192, 32 / 4 heads: 458 and 446);
        // with 256 a wave takes all of a SIMD's registers.
        p.waves = dim != 128 || most <= 128 ? 4 : 8;
        // Blocks that the GPU holds at once (kv_attn_tile.hip: registers allow two
        // waves a SIMD, three of 64 channels, one of 256).  Where there are less
        // than half of them, the keys of each tile are split over blocks (64 tokens
        // over 32768 keys, 64 / 8 heads: 85 us and 12 of the join, unsplit 882).
        // Keys are the table's, the lengths being on the GPU: with one 131072 wide
        // 5 x 64 tokens over 300 .. 600 keys take 25 and 9 us, with one as wide as
        // the longest 27 and 7.  16 splits at the most leave CUs idle where a long
        // context has few tiles of rows (48 heads on one key head, one token over
        // 131072 keys: 16 blocks, 254 and 10 us).
        const int64_t slots = kCus * (dim == 64 ? 3 : dim == 128 && p.waves == 4 ? 2 : 1);
        const int64_t tiles = (T * group + 32 * p.waves - 1) / (32 * p.waves) * heads;
        int64_t splits = slots / tiles;
        if (splits > (keys + 511) / 512) splits = (keys + 511) / 512;
        p.splits = (int)(splits > 16 ? 16 : splits < 1 ? 1 : splits);
        p.tile_parts = (p.bytes + 255) & ~(size_t)255;
        if (p.splits > 1) p.bytes = p.tile_parts + (size_t)p.splits * T * q_heads * (dim + 2) * sizeof(float);
    }
    return p;
}

size_t kv_attention_workspace(int64_t T, int q_heads, int heads, int dim, int fmt, int B, int64_t keys,
                              int64_t max_q) {
    return plan_attention(T, q_heads, heads, dim, fmt, B, keys, max_q).bytes;
}

template <int D, int FMT, int DT, int NT>
static void launch_attn(const KvAttention &a, const Plan &p, hipStream_t stream) {
    kv_attn_kernel<D, FMT, DT, NT><<<(unsigned)p.blocks, 256, 0, stream>>>(a, p.rows_max, a.table);
    if (p.blocks > 1)
        // (a block a row; beside the tile kernel most blocks have nothing to join)
        kv_join_kernel<D, DT, NT><<<dim3((unsigned)p.blocks, p.waves ? 1 : p.rows_max), 256, 0, stream>>>(a);
}

template <int D, int FMT, int DT>
static void launch_attn_nt(const KvAttention &a, const Plan &p, hipStream_t stream) {
    if constexpr (D < 256) {
        if (p.nt == 2) return launch_attn<D, FMT, DT, 2>(a, p, stream);
    }
    launch_attn<D, FMT, DT, 1>(a, p, stream);
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
    const Plan p = plan_attention(a.T, a.q_heads, a.cache.heads, a.cache.dim, a.cache.fmt, a.B,
                                  a.width << a.cache.page_log, max_q);
    if (p.nt) {
        if (a.cache.dim == 64) launch_attn_d<64>(a, p, dt, stream);
        else if (a.cache.dim == 128) launch_attn_d<128>(a, p, dt, stream);
        else launch_attn_d<256>(a, p, dt, stream);
    }
    if (p.waves)
        launch_kv_tiles(a, dt, p.waves, p.rows_max + 1, p.splits,
                        reinterpret_cast<float *>((char *)a.work + p.tile_parts), stream);
}

}  // namespace sq
