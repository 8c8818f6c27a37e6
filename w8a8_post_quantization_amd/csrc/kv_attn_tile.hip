// Attention over the microscaled cache, many queries a sequence (include/
// sq_kv.h): kv_attn.hip's arithmetic and orientation with matrix instructions
// of 32 x 32 x 16, and the keys and values of a tile converted once for a
// block and shared through LDS.
//
// A block takes 32 rows a wave (a row: a query of one of the heads that share
// the key head) over its keys in tiles of 128 (64 with 256 channels).  In LDS
// keys lie [key][channel], values [channel][key], both so that an operand is
// one 16-byte read; the values' keys are in the order in which the weights lie
// in the lanes.  Chunks of 16 bytes are exchanged by an xor with the row's
// number, so that the lanes of a read take all banks.
//
// The matrix cores, LDS (a wave reads every key and value for its 32 rows) and
// the softmax's vector instructions are about equally loaded, so a wave's loop
// overlaps them.  It goes in units of 32 keys: while the scores of the next
// unit are multiplied the weights of this one are formed; while those multiply
// the values, a part of the next tile is converted into LDS and the next
// scores' maximum is taken.  Operands are read from LDS half a unit ahead.  Keys
// and values have two slots in LDS each, with two barriers a tile.
//
// A prompt of 8192, 64 / 8 heads of 128, e2m1, 1.1 TFLOP: 2.4 million cycles,
// which are 1207 .. 1313 us under the profiler (2.01 .. 1.86 GHz) and 1075 ..
// 1095 without, 0.84 .. 1.02 PFLOP/s (a library product of 8192^3 in bf16 1.21);
// e4m3 1285 and fp16 1283 where it took 1250.  The matrix cores are busy 46 % of
// the cycles, the vector units 53 %, LDS 36 %.  Four waves of 64 rows, which read
// LDS half as often, took 2222.  8192 tokens of 32 / 4 heads of 64: 403 .. 469
// us, of 16 / 4 heads of 256: 824 .. 921.
#include <type_traits>

#include "kv_attn_device.h"

namespace sq {

// Where chunk `ch` (16 bytes) of key `key`, and of channel `d`, lies in a slot
// (of KT keys).  LDS moves 256 bytes a clock, 16 lanes of a read: rows of 256
// bytes and more exchange their chunks 16 ways, rows of 128 bytes lie in pairs
// and exchange 8 ways.  Staging writes one channel in D / 16 at a time, so the
// values' exchange takes the higher bits of the channel, too.
template <int D>
__device__ __forceinline__ int key_chunk(int key, int ch) {
    return key * (D / 8) + (ch ^ (D == 64 ? key >> 1 & 7 : key & 15));
}
template <int D, int KT>
__device__ __forceinline__ int value_exchange(int d) {
    constexpr int kPart = D == 64 ? 2 : D == 128 ? 3 : 4;  // log2(D / 16)
    return KT == 128 ? (d ^ d >> kPart) & 15 : (d >> 1 ^ d >> kPart) & 7;
}
template <int D, int KT>
__device__ __forceinline__ int value_chunk(int d, int ch) { return d * (KT / 8) + (ch ^ value_exchange<D, KT>(d)); }

// The order of what follows the last scheduling barrier: a matrix instruction,
// N vector instructions, R times.
template <int R, int N>
__device__ __forceinline__ void mfma_with() {
    if constexpr (R > 0) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, N, 0);
        mfma_with<R - 1, N>();
    }
}

template <int D, int FMT, int DT, int NW>
__global__ __launch_bounds__(64 * NW, D == 64 ? 3 : D == 128 ? 2 : 1) void kv_tile_kernel(const KvAttention a, int rows_min, int splits,
                                                         float *parts, const int32_t *__restrict__ tables) {
    constexpr int NB = D / 32, S = D / 16, JT = D / 32, R = 32 * NW;
    constexpr int KT = D < 256 && NW == 8 ? 128 : 64, UNITS = KT / 32, NT = 64 * NW;  // keys, units of a tile; threads
    static_assert(4 * KT == NT, "a tile is staged by all threads once");
    constexpr int RB = FMT == E2M1 ? D / 2 : D;
    // As a thread stages a tile: of one key a quarter of the channels, and of
    // four successive keys a sixteenth of the values' channels.
    constexpr int KN = RB / 4, KC = D / 4;     // code bytes and channels of a key
    constexpr int KS = KC < 32 ? 1 : KC / 32;  // and scale bytes
    constexpr int VN = RB / 16, VC = D / 16;
    constexpr int SLOT = KT * D / 8;  // chunks of 16 bytes
    __shared__ __attribute__((aligned(1024))) uint4 s_kv[4 * SLOT];
    __shared__ int s_pre[NT + 1], s_wave[NW], s_at[2];
    __shared__ uint32_t s_apart[2][UNITS];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n32 = lane & 31, hh = lane >> 5;
    const int heads = a.cache.heads, plog = a.cache.page_log, group = a.group;

    // The block's rows: tiles of all long sequences in a row, the last (with the
    // most keys) first.
    const auto tiles_of = [&](const KvSeq &s) SQ_INLINE -> int {
        const int64_t rows = (int64_t)s.nq * group;
        return rows < rows_min ? 0 : (int)((rows + R - 1) / R);
    };
    const int per_thread = (a.B + NT - 1) / NT;
    const int b_first = tid * per_thread;
    {
        int sum = 0;
        for (int i = 0; i < per_thread && b_first + i < a.B; ++i) sum += tiles_of(kv_seq(a, b_first + i));
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int v = __shfl_up(sum, off, 64);
            if (lane >= off) sum += v;
        }
        if (lane == 63) s_wave[wave] = sum;
        __syncthreads();
        for (int w = 0; w < wave; ++w) sum += s_wave[w];
        s_pre[tid + 1] = sum;
        if (tid == 0) s_pre[0] = 0;
        __syncthreads();
    }
    // (blocks of no tile are the last: among others they would upset the
    // distribution over the CUs, 150 us for 86 with every third block empty)
    const int want = s_pre[NT] - 1 - (int)(blockIdx.x / (heads * splits));
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
    const int h = blockIdx.x % heads, split = blockIdx.x / heads % splits;
    const KvSeq seq = kv_seq(a, b);
    const int rows = seq.nq * group;  // (T * q_heads < 2^31)

    // Keys that the rows from r to e - 1 see: all of them, any of them.
    const auto span = [&](int r, int e, int &all_lo, int &all_hi, int &any_lo, int &any_hi) SQ_INLINE {
        const int p0 = seq.nk - seq.nq + r / group, p1 = seq.nk - seq.nq + (e - 1) / group;
        any_hi = a.causal ? (p1 + 1 > 0 ? p1 + 1 : 0) : seq.nk;
        all_hi = a.causal ? p0 + 1 : seq.nk;
        any_lo = a.window && (int64_t)p0 - a.window + 1 > 0 ? (int)(p0 - a.window + 1) : 0;
        all_lo = a.window && (int64_t)p1 - a.window + 1 > 0 ? (int)(p1 - a.window + 1) : 0;
    };
    const int r_first = tile * R, r_end = r_first + R < rows ? r_first + R : rows;
    int t_all_lo, t_all_hi, t_lo, t_hi;
    span(r_first, r_end, t_all_lo, t_all_hi, t_lo, t_hi);
    const int w_first = r_first + wave * 32;
    const int w_end = w_first + 32 < rows ? w_first + 32 : rows;
    int w_all_lo = 0, w_all_hi = 0, w_lo = 0, w_hi = 0;
    if (w_first < rows) span(w_first, w_end, w_all_lo, w_all_hi, w_lo, w_hi);

    uint4 qf[S];
    const int row = w_first + n32;  // the lane's
    const int query = row / group;
    const char *const q_row = (const char *)a.q + ((int64_t)(seq.q0 + query) * a.q_st +
                                                   (int64_t)(h * group + row - query * group) * a.q_sh) * 2;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        qf[s] = make_uint4(0, 0, 0, 0);
        if (row < rows) qf[s] = reinterpret_cast<const uint4 *>(q_row)[2 * s + hh];
        if (a.scale < 0) {
            qf[s].x ^= 0x80008000u;
            qf[s].y ^= 0x80008000u;
            qf[s].z ^= 0x80008000u;
            qf[s].w ^= 0x80008000u;
        }
    }
    const int place = seq.nk - seq.nq + query;
    const int r_hi = row < rows ? (a.causal ? place + 1 : seq.nk) : 0;
    const int r_lo = a.window && (int64_t)place - a.window + 1 > 0 ? (int)(place - a.window + 1) : 0;

    float m = kNoMax, l = 0.0f;
    f32x16 o[JT];
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[j][i] = 0.0f;

    // The split's tiles of keys.
    const int t_base = t_lo & ~(KT - 1);
    const int n_all = t_hi > t_lo ? (t_hi - t_base + KT - 1) / KT : 0;
    const int k0 = (int)((int64_t)n_all * split / splits), k1 = (int)((int64_t)n_all * (split + 1) / splits);
    const int n_tiles = k1 - k0;
    // Scores are multiplied by c > 0 as their weights are formed, in one operation
    // with the maximum's subtraction (a negative scale turns the queries), behind
    // hiding and maximum.  Where that does not serve they are multiplied earlier,
    // and c is 1: with a scale of 0, as a hidden score of -inf would turn NaN; and
    // once a row's maximum passes 2^20, since it is rounded and the product is not,
    // so that a weight is 2^(half fp32's step there) off.
    const float to_log2 = fabsf(a.scale) * 1.44269504088896341f;
    constexpr float kEarly = 1048576.0f;
    bool early = to_log2 == 0.0f;
    const auto factor = [&]() SQ_INLINE { return early ? 1.0f : to_log2; };  // c
    const int32_t *const table = tables + (int64_t)b * a.width;
    const int g_last = (t_hi - 1) >> 4;

    // Loads of a tile into registers; tiles past the last are the last again.
    const int sk = tid >> 2, sc = tid & 3, sq4 = tid >> 4, sn = tid & 15;
    Words<KN> rk;
    uint32_t rks[KS];
    Words<VN> rv[4];
    uint32_t rvs[4];
    uint32_t nan_k, nan_v;  // 255 where the page is not in the cache
    int page_k, page_v;     // of the next tile to load
    const auto tile_at = [&](int i) SQ_INLINE { return t_base + (k0 + (i < n_tiles ? i : n_tiles - 1)) * KT; };
    const auto group_of = [&](int key) SQ_INLINE { return key >> 4 < g_last ? key >> 4 : g_last; };
    const auto page_of = [&](int key) SQ_INLINE { return table[group_of(key) >> (plog - 4)]; };
    const auto row_of = [&](int key, int page, uint32_t &nan) SQ_INLINE -> int64_t {
        const bool held = page >= 0 && page < a.cache.pages;
        nan = held ? 0u : 255u;
        return kv_row(a.cache, held ? page : 0, h, ((group_of(key) & ((1 << (plog - 4)) - 1)) << 4) + (key & 15));
    };
    const auto load_keys = [&](int i) SQ_INLINE {
        const int64_t at = row_of(tile_at(i) + sk, page_k, nan_k);
        rk = load_codes<KN>(a.cache.kq + at * RB + sc * KN);
#pragma unroll
        for (int z = 0; z < KS; ++z) rks[z] = a.cache.ks[at * NB + sc * KC / 32 + z];
        page_k = page_of(tile_at(i + 1) + sk);
    };
    const auto load_values = [&](int i) SQ_INLINE {
        const int64_t at = row_of(tile_at(i) + 4 * sq4, page_v, nan_v);
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            rv[z] = load_codes<VN>(a.cache.vq + (at + z) * RB + sn * VN);
            rvs[z] = a.cache.vs[(at + z) * NB + sn * VC / 32];
        }
        page_v = page_of(tile_at(i + 1) + 4 * sq4);
    };
    // In LDS a lane's place is kept as one base, and its other places formed
    // from it as they are needed (exchanged by constants, at constant distances):
    // the compiler is kept from holding them all.
    constexpr int KROW = D * 2, VROW = KT * 2, SLOTB = SLOT * 16;
    uint8_t *const lds = reinterpret_cast<uint8_t *>(s_kv);
    const auto place_of = [&](uint32_t base, int slot) SQ_INLINE {
        base += slot * SLOTB;
        asm("" : "+v"(base));
        return base;
    };
    const uint32_t to_k = 16 * key_chunk<D>(sk, sc * (KC / 8));
    const uint32_t to_v = 2 * SLOTB + 16 * value_chunk<D, KT>(sn * VC, (sq4 >> 2) * 2 + (sq4 & 1)) + 8 * ((sq4 & 3) >> 1);
    const auto stage_keys = [&](int slot) SQ_INLINE {
        const uint32_t to = place_of(to_k, slot);
#pragma unroll
        for (int z = 0; z < KC / 8; ++z) {
            const float s = e8m0(rks[KC < 32 ? 0 : z / 4] | nan_k);
            *reinterpret_cast<uint4 *>(lds + (to ^ 16 * z)) = codes8_to_16<FMT, DT>(&rk.w[z * (FMT == E2M1 ? 1 : 2)], s);
        }
    };
    const auto stage_values = [&](int i, int slot) SQ_INLINE {
        const int t = tile_at(i);
#pragma unroll
        for (int z = 0; z < 4; ++z) rvs[z] |= nan_v;
        if (t < t_all_lo || t + KT > t_all_hi) {
            asm volatile("");  // (a branch, not selects)
            // Keys that no row of the block sees (behind the last, before the
            // window) are taken as 0: what their place holds may be anything.
            // Where an infinity or NaN may be, it is set apart: a weight of 0
            // does not keep it from a row that must not see it.
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const int key = 4 * sq4 + z;
                const bool none = t + key < t_lo || t + key >= t_hi;
                const bool alone = !none && may_be_nonfinite<FMT, DT>(rv[z], rvs[z]);
                if (alone) atomicOr(&s_apart[slot][key >> 5], 1u << (key & 31));
                if (none || alone) {
                    rv[z] = Words<VN>{};
                    rvs[z] = 0;
                }
            }
        }
        // (in a group of 16 keys the quads lie 0, 2, 1, 3)
        const uint32_t to = place_of(to_v, slot);
        float s[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) s[z] = e8m0(rvs[z]);
#pragma unroll
        for (int q = 0; q < VC / 2; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) w[z] = pair_of<FMT, DT>(rv[z], q, s[z]);
#pragma unroll
            for (int odd = 0; odd < 2; ++odd) {
                const int c = 2 * q + odd, x = KT == 128 ? c : c >> 1;
                const uint32_t sel = odd ? 0x07060302u : 0x05040100u;
                *reinterpret_cast<uint2 *>(lds + (to ^ 16 * x) + c * VROW) =
                    make_uint2(__builtin_amdgcn_perm(w[1], w[0], sel), __builtin_amdgcn_perm(w[3], w[2], sel));
            }
        }
    };

    // Scores of 32 keys, their largest, the weights, the weighted values.
    struct Weights { u4v p[2]; };
    // Operands: chunk 2 s + hh of key 32 sub + n32, chunk 4 sub + 2 u + hh of
    // channel 32 j + n32.
    const uint32_t at_k = 16 * key_chunk<D>(n32, hh), at_v = 2 * SLOTB + 16 * value_chunk<D, KT>(n32, hh);
    const auto read_keys = [&](uint4 (&f)[S], int slot, int sub, int from, int to) SQ_INLINE {
        const uint32_t at = place_of(at_k, slot);
#pragma unroll
        for (int s = from; s < to; ++s)
            f[s] = *reinterpret_cast<const uint4 *>(lds + (at ^ 32 * (s & 7)) + sub * 32 * KROW + (s & ~7) * 32);
    };
    const auto read_values = [&](uint4 (&f)[JT], int slot, int sub, int u) SQ_INLINE {
        const uint32_t at = place_of(at_v, slot);
#pragma unroll
        for (int j = 0; j < JT; ++j) {
            const int x = (4 * sub + 2 * u ^ value_exchange<D, KT>(32 * j)) & (KT / 8 - 1);
            f[j] = *reinterpret_cast<const uint4 *>(lds + (at ^ 16 * x) + j * 32 * VROW);
        }
    };
    const auto multiply_keys = [&](f32x16 &x, const uint4 (&f)[S]) SQ_INLINE {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 0.0f;
#pragma unroll
        for (int s = 0; s < S; ++s) x = mfma32<DT>(f[s], qf[s], x);
    };
    const auto multiply_values = [&](const u4v &w, const uint4 (&f)[JT]) SQ_INLINE {
#pragma unroll
        for (int j = 0; j < JT; ++j) o[j] = mfma32<DT>(f[j], make_uint4(w.x, w.y, w.z, w.w), o[j]);
    };
    const auto hide = [&](f32x16 &x, int t) SQ_INLINE {
        if (early || t < w_all_lo || t + 32 > w_all_hi) {
            asm volatile("");  // (a branch, not selects)
            if (early) x *= to_log2;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int key = t + (i & 3) + 8 * (i >> 2) + 4 * hh;
                if (key < r_lo || key >= r_hi) x[i] = -INFINITY;
            }
        }
    };
    const auto largest = [&](const f32x16 &x) SQ_INLINE {
        float top = x[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, x[i]);
        return top * factor();
    };
    // Rows are rescaled only where the maximum trails by more than it may.
    const auto rescale = [&](f32x16 &x, float top) SQ_INLINE {
        if (__any(top - m > kTrail + kLift<DT>)) {
            const float mn = fmaxf(m, fmaxf(top, __shfl_xor(top, 32, 64)) - kLift<DT>);
            const float f = __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= f;
#pragma unroll
            for (int j = 0; j < JT; ++j) o[j] *= f;
            if (!early && __any(fabsf(mn) > kEarly && mn != kNoMax)) {
                early = true;
                x *= to_log2;
            }
        }
    };
    const auto form_weights = [&](f32x16 &x, Weights &w) SQ_INLINE {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], factor(), -m));
            l += x[i];
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
            w.p[u] = u4v{pack16<DT>(x[8 * u], x[8 * u + 1]), pack16<DT>(x[8 * u + 2], x[8 * u + 3]),
                         pack16<DT>(x[8 * u + 4], x[8 * u + 5]), pack16<DT>(x[8 * u + 6], x[8 * u + 7])};
    };
    // (rare) The keys set apart, one at a time, for the rows that see them.
    const auto add_apart = [&](const Weights &w, int t, uint32_t keys) SQ_INLINE {
        for (; keys; keys &= keys - 1) {
            const int n = __builtin_ctz(keys), key = t + n;
            const int i = (n & 3) + 4 * (n >> 3), from = n32 + 32 * (n >> 2 & 1);
            const int page = page_of(key);
            const bool held = page >= 0 && page < a.cache.pages;
            const int64_t at_row = kv_row(a.cache, held ? page : 0, h, key & ((1 << plog) - 1));
            const uint32_t words[8] = {w.p[0].x, w.p[0].y, w.p[0].z, w.p[0].w, w.p[1].x, w.p[1].y, w.p[1].z, w.p[1].w};
            uint32_t pair = words[0];
#pragma unroll
            for (int z = 1; z < 8; ++z) pair = z == i >> 1 ? words[z] : pair;
            const float p = __shfl(half_of<DT>(pair, i & 1), from, 64);
#pragma unroll
            for (int j = 0; j < JT; ++j)
#pragma unroll
                for (int z = 0; z < 4; ++z) {  // channels d .. d + 3, of one staged part
                    const int d = 32 * j + 8 * z + 4 * hh;
                    const Words<VN> v = load_codes<VN>(a.cache.vq + at_row * RB + d / VC * VN);
                    const uint32_t e = held ? a.cache.vs[at_row * NB + j] : 255u;
                    if (!may_be_nonfinite<FMT, DT>(v, e)) continue;  // (not set apart)
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        float val = 0.0f;
#pragma unroll
                        for (int at = 0; at < VC; at += 4)
                            if (d % VC == at) val = half_of<DT>(pair_of<FMT, DT>(v, (at + y) >> 1, e8m0(e)), y & 1);
                        if (key >= r_lo && key < r_hi) o[j][4 * z + y] += p * val;
                    }
                }
        }
    };

    if (tid < 2 * UNITS) s_apart[tid / UNITS][tid % UNITS] = 0;
    if (n_tiles > 0) {
        page_k = page_of(tile_at(0) + sk);
        page_v = page_of(tile_at(0) + 4 * sq4);
        load_keys(0);
        load_values(0);
        __syncthreads();  // (s_apart)
        stage_keys(0);
        stage_values(0, 0);
        load_keys(1);
        load_values(1);
        __syncthreads();
        f32x16 x[2];
        Weights w;
        uint4 kf[S], vf[2][JT];
        read_keys(kf, 0, 0, 0, S);
        multiply_keys(x[0], kf);
        read_keys(kf, 0, 1, 0, S / 2);
        hide(x[0], tile_at(0));
        rescale(x[0], largest(x[0]));
        wait_vmcnt<0>();  // (else the queries' loads count as pending in the loop)
        for (int i = 0; i < n_tiles; ++i) {
            const int t = tile_at(i), slot = i & 1;
            uint32_t apart[UNITS];  // the tile's keys set apart
            // Unit u of the tile is weighted, the next one (whose keys' operands
            // are read) scored, and the operands of the one after it read.
            const auto unit = [&](auto number) SQ_INLINE {
                constexpr int u = decltype(number)::value;
                constexpr bool last = u == UNITS - 1;
                read_keys(kf, last ? slot ^ 1 : slot, (u + 1) % UNITS, S / 2, S);
                read_values(vf[0], slot, u, 0);
                __builtin_amdgcn_sched_barrier(0);
                multiply_keys(x[~u & 1], kf);
                form_weights(x[u & 1], w);
                // (kept here: the compiler would move the weights behind the branches)
                asm volatile("" : "+v"(w.p[0]), "+v"(w.p[1]), "+v"(l));
                mfma_with<S, 56 / S>();
                __builtin_amdgcn_sched_barrier(0);
                hide(x[~u & 1], last ? tile_at(i + 1) : t + 32 * (u + 1));
                read_values(vf[1], slot, u, 1);
                multiply_values(w.p[0], vf[0]);
                if constexpr (u == 0) {
                    stage_keys(slot ^ 1);
                    load_keys(i + 2);
                    if (tid < UNITS) s_apart[slot ^ 1][tid] = 0;
                }
                if constexpr (u == (UNITS == 4 ? 2 : 1)) {
                    stage_values(i + 1, slot ^ 1);
                    load_values(i + 2);
                }
                // The first barrier stands between the staging of the next keys
                // and their reading, the second the values'; either also between
                // the last reads of a slot and its staging.
                if constexpr (u == 0 || u == (UNITS == 4 ? 2 : 1)) lds_barrier();
                read_keys(kf, u + 2 < UNITS ? slot : slot ^ 1, (u + 2) % UNITS, 0, S / 2);
                // (all units' at once: between the tile's second barrier and the
                // next one's first they are cleared)
                if constexpr (u == 0) {
#pragma unroll
                    for (int z = 0; z < UNITS; ++z) apart[z] = __builtin_amdgcn_readfirstlane(s_apart[slot][z]);
                }
                multiply_values(w.p[1], vf[1]);
                const float top = largest(x[~u & 1]);
                if (apart[u]) {
                    add_apart(w, t + 32 * u, apart[u]);
                    // (loads of it that are left unused would be waited for below,
                    // whether it ran or not)
                    wait_vmcnt<0>();
                }
                rescale(x[~u & 1], top);
            };
            unit(std::integral_constant<int, 0>{});
            unit(std::integral_constant<int, 1>{});
            if constexpr (UNITS == 4) {
                unit(std::integral_constant<int, 2>{});
                unit(std::integral_constant<int, 3>{});
            }
        }
    }

    l += __shfl_xor(l, 32, 64);
    if (row >= rows) return;
    const int64_t out = (int64_t)(seq.q0 + query) * a.q_heads + h * group + row - query * group;
    if (splits == 1) {
        const float inv = row_factor(l, r_hi, seq.over);
        uint2 *y = reinterpret_cast<uint2 *>(a.y) + out * (D / 4) + hh;
#pragma unroll
        for (int j = 0; j < JT; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                y[8 * j + 2 * k] = make_uint2(pack16<DT>(o[j][4 * k] * inv, o[j][4 * k + 1] * inv),
                                              pack16<DT>(o[j][4 * k + 2] * inv, o[j][4 * k + 3] * inv));
    } else {
        // values of all rows and splits, then their maxima and sums
        const int64_t all = (int64_t)a.T * a.q_heads;
        float *y = parts + (split * all + out) * D + 4 * hh;
#pragma unroll
        for (int j = 0; j < JT; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                *reinterpret_cast<float4 *>(y + 32 * j + 8 * k) =
                    make_float4(o[j][4 * k], o[j][4 * k + 1], o[j][4 * k + 2], o[j][4 * k + 3]);
        if (hh == 0) {
            float *s = parts + splits * all * D + (split * all + out) * 2;
            s[0] = m;
            s[1] = l;
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
    const float inv = row_factor(sum, keys_end(a, seq, t - seq.q0), seq.over);
    reinterpret_cast<uint2 *>(a.y)[row * Q + d4] =
        make_uint2(pack16<DT>(v[0] * inv, v[1] * inv), pack16<DT>(v[2] * inv, v[3] * inv));
}

template <int D, int FMT, int DT, int NW>
static void launch_tile(const KvAttention &a, int rows_min, int splits, float *parts, hipStream_t stream) {
    // (whatever the sequences' lengths: each leaves its last tile open at the most)
    const int64_t open = a.B < a.T ? a.B : a.T, tiles = (a.T * a.group + open * (32 * NW - 1)) / (32 * NW);
    kv_tile_kernel<D, FMT, DT, NW><<<(unsigned)(tiles * a.cache.heads * splits), 64 * NW, 0, stream>>>(
        a, rows_min, splits, parts, a.table);
    if (splits > 1) {
        const int64_t rows = a.T * a.q_heads, per = 256 / (D / 4);
        kv_tile_join_kernel<D, DT><<<(unsigned)((rows + per - 1) / per), 256, 0, stream>>>(a, rows_min, splits, parts);
    }
}

template <int D, int FMT, int DT>
static void launch_tile_nw(const KvAttention &a, int waves, int rows_min, int splits, float *parts,
                           hipStream_t stream) {
    if constexpr (D == 128) {
        if (waves == 8) return launch_tile<D, FMT, DT, 8>(a, rows_min, splits, parts, stream);
    }
    launch_tile<D, FMT, DT, 4>(a, rows_min, splits, parts, stream);
}

template <int D>
static void launch_tile_d(const KvAttention &a, int dt, int waves, int rows_min, int splits, float *parts,
                          hipStream_t stream) {
    if (a.cache.fmt == E2M1) {
        if (dt == F16) launch_tile_nw<D, E2M1, F16>(a, waves, rows_min, splits, parts, stream);
        else launch_tile_nw<D, E2M1, BF16>(a, waves, rows_min, splits, parts, stream);
    } else {
        if (dt == F16) launch_tile_nw<D, E4M3, F16>(a, waves, rows_min, splits, parts, stream);
        else launch_tile_nw<D, E4M3, BF16>(a, waves, rows_min, splits, parts, stream);
    }
}

void launch_kv_tiles(const KvAttention &a, int dt, int waves, int rows_min, int splits, float *parts,
                     hipStream_t stream) {
    if (a.cache.dim == 64) launch_tile_d<64>(a, dt, waves, rows_min, splits, parts, stream);
    else if (a.cache.dim == 128) launch_tile_d<128>(a, dt, waves, rows_min, splits, parts, stream);
    else launch_tile_d<256>(a, dt, waves, rows_min, splits, parts, stream);
}

}  // namespace sq
