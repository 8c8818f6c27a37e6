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
//
// Two kernels:
//  * mx_gemm_dec  M <= 32 (decode), bound by the weight stream; also K < 256,
//                 bound by the outputs' stores.
//  * mx_gemm_pp   M > 32: both operands through LDS rings filled by
//                 direct-to-LDS loads.
#include <type_traits>

#include "mx_device.h"
#include "pipe_device.h"
#include "sq_launch.h"

namespace sq {

struct MxArgs : TileGrid {
    const uint8_t *xq, *xs, *wq, *ws;
    int M, N, K;
    void *y;
    int y_dt;
    int groups;  // mx_gemm_dec: groups of 16 weight rows a block covers (tiles_n blocks over N)
};

__device__ __forceinline__ int8x lo128(int4v a) {  // an e2m1 operand: the upper half is not read
    return __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
}
__device__ __forceinline__ int8x both128(int4v a, int4v b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// An activation fragment: one 16-byte chunk a lane (e2m1) or two (e4m3).
template <int XF> struct XFrag { int4v c[XF == E4M3 ? 2 : 1]; };
template <int XF>
__device__ __forceinline__ int8x operand(const XFrag<XF> &f) {
    if constexpr (XF == E4M3) return both128(f.c[0], f.c[1]);
    else return lo128(f.c[0]);
}

// e4m3 activations multiply in two parts, |x| >= 2 and |x| < 2, by an
// instruction each (kParts).  With an e4m3 operand the instruction aligns the
// products of eight successive k to the largest exponent among them and drops
// what lies below 2^-13 of it, in all up to 2^-10.7 of a step's largest product
// (measured); the groups of eight it adds as exactly as with e2m1.  The products
// of one part stay above that: multiples of 2^-3 with exponents up to 10 where
// |x| >= 2, of 2^-10 up to 2 where |x| < 2.  So a step is exact where its blocks'
// scales are equal and else within 2^-20 of its largest product (measured: worst
// 2^-20.4 over scales 2^+-20), as with e2m1.
// It costs a second MFMA where these bound the kernel: 256 x 28672 x 7168 57 us
// in one part and 87 in two, 4096 x 14336 x 4096 212 and 317, 2048 x 4096 x 4096
// 33 and 46; 1 x 28672 x 8192 23.9 and 24.7, 32 tokens 30.5 and 32.9.  One part
// would leave an fp32 sum off by 3.5 10^-5 and 16-bit outputs by 1 to 5 10^-4,
// beside an own rounding of 2 (fp16) and 17 10^-4 (bf16).
template <int XF> constexpr int kParts = XF == E4M3 ? 2 : 1;

// Four codes' part P: 0 those with |x| >= 2 (bit 6 of the byte set), 1 the
// others; zero in place of the rest.
template <int P>
__device__ __forceinline__ int part4(int v) {
    // a byte permute whose selectors 8 .. 11 spread the sign bit of an odd byte
    const uint32_t m = __builtin_amdgcn_perm((uint32_t)v << 9, (uint32_t)v << 1, 0x090b080au);
    return (int)(P == 0 ? (uint32_t)v & m : (uint32_t)v & ~m);
}
template <int XF, int P>
__device__ __forceinline__ XFrag<XF> part_of(const XFrag<XF> &f) {
    XFrag<XF> r = f;
    if constexpr (XF == E4M3) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) r.c[c][i] = part4<P>(f.c[c][i]);
    }
    return r;
}

template <int XF>
__device__ __forceinline__ void set_parts(XFrag<XF> (&p)[kParts<XF>], const XFrag<XF> &f) {
    p[0] = part_of<XF, 0>(f);
    if constexpr (kParts<XF> == 2) p[1] = part_of<XF, 1>(f);
}

// One scaled product; Q: the byte of the scale registers that applies.
template <int XF, int Q>
__device__ __forceinline__ f32x16 mfma32(int4v w, const XFrag<XF> &x, f32x16 acc, int sw, int sx) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(lo128(w), operand<XF>(x), acc, 4,
                                                           XF == E4M3 ? 0 : 4, Q, sw, Q, sx);
}
template <int XF, int Q>
__device__ __forceinline__ f32x4 mfma16(int4v w, const XFrag<XF> &x, f32x4 acc, int sw, int sx) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(lo128(w), operand<XF>(x), acc, 4,
                                                            XF == E4M3 ? 0 : 4, Q, sw, Q, sx);
}

// ---------------------------------------------------------------- tiled

// Outputs of a wave's accumulators (32x32 layout: lane l, register v of
// fragment (i, j) is weight row 8 (v / 4) + 4 (l / 32) + v % 4 of n-fragment
// i, token l % 32 of m-fragment j) through a wave-private slab of LDS: 32
// token rows of the output type per m-fragment, read back 16 bytes a lane
// along rows, so that stores cover 128 to 512 contiguous bytes of a row.
// 16-byte chunk c of slab row r sits at position c ^ f(r).
template <int BM, int BN, int WM, int WN, int YDT>
__device__ __forceinline__ void mx_epilogue(const MxArgs &p,
                                            f32x16 (&acc)[BN / WN / 32][BM / WM / 32],
                                            uint8_t *smem, int m0, int n0) {
    constexpr int WTM = BM / WM, WTN = BN / WN;
    constexpr int FM = WTM / 32, FN = WTN / 32;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / WN, wn = wave % WN;
    const int fr = lane & 31, fh = lane >> 5;
    const int M = p.M, N = p.N;
    using T = typename OutT<YDT>::T;
    constexpr int RB = WTN * (int)sizeof(T);       // slab row bytes
    constexpr int CPR = RB / 16;                   // 16-byte chunks per row
    constexpr int RPW = RB >= 256 ? 1 : 256 / RB;  // rows per 256-byte bank window
    constexpr int EPC = 16 / (int)sizeof(T);       // outputs per chunk
    static_assert(RB % 16 == 0 && (32 * CPR) % 64 == 0, "slab");
    uint8_t *slab = smem + wave * (32 * RB);
    const bool vec_y = N % EPC == 0 && ((uintptr_t)p.y & 15) == 0;
#pragma unroll
    for (int j = 0; j < FM; ++j) {
        const int fw = (fr / RPW) & (CPR - 1);
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                T h[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) h[q] = narrow<YDT>(acc[i][j][4 * g + q]);
                const int cb = (i * 32 + 8 * g + 4 * fh) * (int)sizeof(T);
                uint8_t *dst = slab + fr * RB + (((cb >> 4) ^ fw) << 4) + (cb & 15);
                if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4 *>(dst) = __builtin_bit_cast(uint4, h);
                else *reinterpret_cast<uint2 *>(dst) = __builtin_bit_cast(uint2, h);
            }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // slab written (one wave)
        if (!vec_y) {
            // rows that start anywhere: successive lanes store successive outputs
#pragma unroll 8
            for (int k = 0; k < 32 * WTN / 64; ++k) {
                const int i = k * 64 + lane, r = i / WTN, nl = i % WTN;
                const int cb = nl * (int)sizeof(T);
                const T v = *reinterpret_cast<const T *>(
                    slab + r * RB + (((cb >> 4) ^ ((r / RPW) & (CPR - 1))) << 4) + (cb & 15));
                const int m = m0 + wm * WTM + j * 32 + r, n = n0 + wn * WTN + nl;
                if (m < M && n < N) reinterpret_cast<T *>(p.y)[(int64_t)m * N + n] = v;
            }
        } else
#pragma unroll
        for (int k = 0; k < 32 * CPR / 64; ++k) {
            const int c = lane + 64 * k;
            const int r = c / CPR, ch = c % CPR;
            const uint4 v = *reinterpret_cast<const uint4 *>(
                slab + r * RB + ((ch ^ ((r / RPW) & (CPR - 1))) << 4));
            const int m = m0 + wm * WTM + j * 32 + r;
            const int n = n0 + wn * WTN + ch * EPC;
            if (m >= M || n >= N) continue;
            T *yp = reinterpret_cast<T *>(p.y) + (int64_t)m * N + n;
            if (n + EPC <= N) {
                // 16-bit outputs past the caches (4096 x 14336 x 4096: 130 us
                // against 136; fp32 ones measured 23.1 us so, 22.5 not)
                if constexpr (sizeof(T) == 2)
                    __builtin_nontemporal_store(__builtin_bit_cast(u4v, v), reinterpret_cast<u4v *>(yp));
                else *reinterpret_cast<uint4 *>(yp) = v;
            } else {
                T e[EPC];
                __builtin_memcpy(e, &v, 16);
#pragma unroll
                for (int q = 0; q < EPC; ++q)
                    if (n + q < N) yp[q] = e[q];
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // slab read before reuse
    }
}

// MQ MFMAs with RQ LDS reads spread between them (a wave issues in order: a
// read queued behind the MFMAs would wait for the matrix core), and after
// the stage barrier the stage's L direct loads too.
template <int MQ, int RQ, int L, int I = 0>
__device__ __forceinline__ void mx_sched() {
    if constexpr (I < MQ) {
        constexpr int R0 = I * RQ / MQ, R1 = (I + 1) * RQ / MQ;
        constexpr int L0 = I * L / MQ, L1 = (I + 1) * L / MQ;
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if constexpr (R1 > R0) __builtin_amdgcn_sched_group_barrier(0x100, R1 - R0, 0);
        if constexpr (L1 > L0) __builtin_amdgcn_sched_group_barrier(0x020, L1 - L0, 0);
        mx_sched<MQ, RQ, L, I + 1>();
    }
}

// K >= 256.  A stage is 256 elements of K: 128 bytes of every weight row and
// 128 (e2m1) or twice 128 (e4m3, two half tiles) of every activation row,
// streamed into a ring of STA LDS stages by direct-to-LDS loads, with chunk c
// of a 128-byte row r at slot c ^ swz(r).  It is consumed as four quarters of
// 64 elements.
//
// Which blocks of a stage meet in a quarter is free as long as both operands
// agree: lane half h takes block 4 h + q in quarter q, so a lane's four scale
// bytes of a stage are one aligned word of the row's eight, and the
// instruction selects byte q (e4m3: the chunks that the instruction pairs
// with blocks q and 4 + q, the file comment).
//
// Scales.  A row's bytes of one stage are 8, and a load of those would cost
// the vector L1 as many line requests as the stage's data (a line per row and
// stage; 256 x 28672 x 7168 e2m1: 47 us so, 44 with CH = 4).  K % 128 == 0
// (CH > 0): the bytes of CH stages are loaded at a time into an LDS area
// beside the ring, read into CH words per fragment when their first stage
// comes up, and the area is refilled during that stage.
// Other K (CH = 0: a scale row starts at any byte, which direct-to-LDS loads
// cannot fetch): each thread loads one row's eight bytes with the stage's
// data and writes them to LDS where the stage is waited for.
//
// K % 256 != 0: the last stage is the row's last 256 elements again, and the
// weights of its first blocks, which are added already, count as zero.
//
// Measured: 4096 x 14336 x 4096 134 us e2m1 (3.6 PFLOP/s; an MFMA loop alone
// reaches 6.3), 317 us e4m3 (1.5, in two parts each of 1.65); 256 x 28672 x 7168
// 41 and 87 us, where e2m1's loads alone take 37 and its products from LDS alone
// 29: the direct loads of both operands share a CU's in-order queue of vector L1
// misses.
template <int XF, int BM, int BN, int WM, int WN, int STA, int CH>
__global__ __launch_bounds__(64 * WM * WN, 2) void mx_gemm_pp(MxArgs p) {
    constexpr bool REGS = CH == 0;
    constexpr int NW = WM * WN, XH = XF == E4M3 ? 2 : 1;
    constexpr int WTM = BM / WM, WTN = BN / WN;
    constexpr int FM = WTM / 32, FN = WTN / 32;
    constexpr int LX = BM * XH / (8 * NW), LW = BN / (8 * NW);  // 1 KB loads per wave and stage
    constexpr int RPS = REGS ? 1 : 32 / (REGS ? 1 : CH);         // rows per 256 B scale load
    constexpr int LS = REGS ? 0 : (BM + BN) / (RPS * NW);        // scale loads per CH stages
    constexpr int L = LX + LW;
    constexpr int SX = BM * 128 * XH, SW = BN * 128, STG = SX + SW;
    constexpr int SS = (BM + BN) * 8 * (REGS ? 2 : CH);
    static_assert(FM >= 1 && FN >= 1 && LX >= 1 && LW >= 1, "tile");
    static_assert(CH == 0 || CH == 2 || CH == 4, "stages per scale load");
    static_assert(REGS || (LS * RPS * NW == BM + BN && BM % RPS == 0 && STA <= CH + 1), "scale loads");
    static_assert(STA >= 2 && STA * L + 2 * LS < 64, "vmcnt range");
    static_assert(!REGS || (BM + BN <= 64 * NW && STA == 2), "a thread per scale row");
    static_assert(NW * 32 * WTN * 4 <= STA * STG, "slabs");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[STA * STG + SS];
    uint8_t *const sscale = smem + STA * STG;

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave / WN, wn = wave % WN;
    int tile_m, tile_n;
    tile_of(p, blockIdx.x, tile_m, tile_n);
    const int m0 = tile_m * BM, n0 = tile_n * BN;
    const int M = p.M, N = p.N, K = p.K;
    const int KB = K >> 5;
    const int nk = (KB + 7) >> 3;
    const int skip = nk * 8 - KB;  // blocks of the last stage that are added already

    // This wave's loads: offsets of its lanes from the tile's first row (rows
    // past the edge read a valid row, whose outputs are never stored).
    uint32_t x_off[LX], w_off[LW];
    const int mtop = M - 1 - m0, ntop = N - 1 - n0;
#pragma unroll
    for (int j = 0; j < LX; ++j) {
        const int b = wave * LX + j, hh = b / (BM / 8), row = (b % (BM / 8)) * 8 + (lane >> 3);
        const int c = (lane & 7) ^ swz(row);
        x_off[j] = (uint32_t)(row < mtop ? row : mtop) * (uint32_t)(K * XH / 2) + hh * 128 + c * 16 +
                   dma_bias<16>(j);
    }
#pragma unroll
    for (int j = 0; j < LW; ++j) {
        const int row = (wave * LW + j) * 8 + (lane >> 3);
        const int c = (lane & 7) ^ swz(row);
        w_off[j] = (uint32_t)(row < ntop ? row : ntop) * (uint32_t)(K / 2) + c * 16 + dma_bias<16>(j);
    }
    const uint8_t *xs0 = p.xs + (int64_t)m0 * KB, *ws0 = p.ws + (int64_t)n0 * KB;
    const uint32_t waveu = (uint32_t)__builtin_amdgcn_readfirstlane(wave);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void_t *)smem;
    const uint8_t *xq0 = p.xq + (int64_t)m0 * (K * (int64_t)XH / 2), *wq0 = p.wq + (int64_t)n0 * (K / 2);
    const uint8_t *s_row = nullptr;  // REGS: this thread's scale row
    if constexpr (REGS) {
        const int t = tid < BM + BN ? tid : BM + BN - 1;  // (spare threads repeat the last row)
        s_row = t < BM ? xs0 + (int64_t)(t < mtop ? t : mtop) * KB
                       : ws0 + (int64_t)(t - BM < ntop ? t - BM : ntop) * KB;
    }
    uint2 rs = make_uint2(0, 0);
    auto issue = [&](int s) __attribute__((always_inline)) {  // stage s < nk
        const uint32_t base = lds0 + (uint32_t)((s % STA) * STG);
        const int b0 = s * 8 < KB - 8 ? s * 8 : KB - 8;  // the stage's first block
        lds_dma_based<LX, 16, false>(x_off, xq0 + b0 * (16 * XH), base + waveu * (LX * 1024u));
        lds_dma_based<LW, 16, false>(w_off, wq0 + b0 * 16, base + SX + waveu * (LW * 1024u));
        if constexpr (REGS) __builtin_memcpy(&rs, s_row + b0, 8);
    };
    // CH > 0: the scales of stages CH c .. CH c + CH - 1.  Load i of the block
    // covers RPS rows of 2 CH words, activation rows first; words past a row's
    // end repeat its last.  Word d of a row sits at d ^ scale_swz(row), which
    // spreads the words that a wave reads (one per row and lane half) over
    // all banks.
    auto scale_swz = [](int row) { return 2 * ((row / RPS) & (32 / RPS - 1)); };
    auto issue_scales = [&](int c) __attribute__((always_inline)) {
        if constexpr (!REGS) {
            // (opaque, so that the offsets below are formed here, every CH
            // stages, and not kept in registers through the loop)
            int ln = lane;
            asm volatile("" : "+v"(ln));
#pragma unroll
            for (int j = 0; j < LS; ++j) {
                const int i = (int)waveu * LS + j;
                const bool is_x = i < BM / RPS;
                const int r = (is_x ? i : i - BM / RPS) * RPS + ln / (2 * CH), top = is_x ? mtop : ntop;
                int b = 8 * CH * c + 4 * ((ln & (2 * CH - 1)) ^ scale_swz(i * RPS));
                b = b < KB - 4 ? b : KB - 4;
                const uint32_t off = (uint32_t)(r < top ? r : top) * (uint32_t)KB + (uint32_t)b + dma_bias<4>(0);
                lds_dma_based<1, 4, false>(&off, is_x ? xs0 : ws0, lds0 + (uint32_t)(STA * STG) + i * 256u);
            }
        }
    };

    const int fr = lane & 31, fh = lane >> 5;
    const int fsw = swz(fr);  // fragment bases are multiples of 32 rows
    auto read_frags = [&](int s, int q, XFrag<XF> (&xf)[FM],
                          int4v (&wf)[FN]) __attribute__((always_inline)) {
        const uint8_t *xb = smem + (s % STA) * STG;
        const uint8_t *wb = smem + (s % STA) * STG + SX;
#pragma unroll
        for (int f = 0; f < FM; ++f)
#pragma unroll
            for (int c = 0; c < XH; ++c) {
                // e4m3: chunk 2 q + h of block q's half tile, then of 4 + q's
                const int ch = XF == E4M3 ? 2 * q + fh : 4 * fh + q;
                xf[f].c[c] = *reinterpret_cast<const int4v *>(
                    xb + c * (BM * 128) + (wm * WTM + f * 32 + fr) * 128 + ((ch ^ fsw) << 4));
            }
#pragma unroll
        for (int f = 0; f < FN; ++f)
            wf[f] = *reinterpret_cast<const int4v *>(wb + (wn * WTN + f * 32 + fr) * 128 +
                                                     (((4 * fh + q) ^ fsw) << 4));
    };
    // A fragment's scale words: [0] the next stage's, then (CH > 0) those of
    // the stages after it that the area held when it was read.
    constexpr int SN = REGS ? 1 : CH;
    uint32_t nx[FM][SN], nw[FN][SN];
    auto read_scales = [&](int s) __attribute__((always_inline)) {  // stage s becomes the next
        if constexpr (REGS) {
            const uint8_t *b = sscale + (s & 1) * ((BM + BN) * 8) + 4 * fh;
#pragma unroll
            for (int f = 0; f < FM; ++f)
                nx[f][0] = *reinterpret_cast<const uint32_t *>(b + (wm * WTM + f * 32 + fr) * 8);
#pragma unroll
            for (int f = 0; f < FN; ++f)
                nw[f][0] = *reinterpret_cast<const uint32_t *>(b + (BM + wn * WTN + f * 32 + fr) * 8);
        } else if ((s & (SN - 1)) == 0) {
            const uint8_t *at[SN];
            int row = fr;
            asm volatile("" : "+v"(row));  // (as in issue_scales)
#pragma unroll
            for (int i = 0; i < SN; ++i) {
                // (the last stage of K % 256 == 128 has its new blocks in its
                // area's first word, and they are the upper lane half's)
                const int d = 2 * i + (skip && s + i == nk - 1 ? 0 : fh);
                at[i] = sscale + row * (8 * SN) + 4 * (d ^ scale_swz(row));
            }
#pragma unroll
            for (int f = 0; f < FM; ++f)
#pragma unroll
                for (int i = 0; i < SN; ++i)
                    nx[f][i] = *reinterpret_cast<const uint32_t *>(at[i] + (wm * WTM + f * 32) * (8 * SN));
#pragma unroll
            for (int f = 0; f < FN; ++f)
#pragma unroll
                for (int i = 0; i < SN; ++i)
                    nw[f][i] = *reinterpret_cast<const uint32_t *>(at[i] + (BM + wn * WTN + f * 32) * (8 * SN));
        } else {
#pragma unroll
            for (int i = 0; i + 1 < SN; ++i) {
#pragma unroll
                for (int f = 0; f < FM; ++f) nx[f][i] = nx[f][i + 1];
#pragma unroll
                for (int f = 0; f < FN; ++f) nw[f][i] = nw[f][i + 1];
            }
        }
    };

    f32x16 acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    int cx[FM], cw[FN];  // this stage's scales
    auto mma = [&](auto qc, const XFrag<XF> (&xf)[FM],
                   const int4v (&wf)[FN]) __attribute__((always_inline)) {
        constexpr int Q = decltype(qc)::value;
        auto with = [&](auto pc) __attribute__((always_inline)) {
            constexpr int P = decltype(pc)::value;
            XFrag<XF> xp[FM];
#pragma unroll
            for (int j = 0; j < FM; ++j) xp[j] = part_of<XF, P>(xf[j]);
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j)
                    acc[i][j] = mfma32<XF, Q>(wf[i], xp[j], acc[i][j], cw[i], cx[j]);
        };
        with(std::integral_constant<int, 0>{});
        if constexpr (kParts<XF> == 2) with(std::integral_constant<int, 1>{});
    };
    auto take_scales = [&]() {
#pragma unroll
        for (int f = 0; f < FM; ++f) cx[f] = (int)nx[f][0];
#pragma unroll
        for (int f = 0; f < FN; ++f) cw[f] = (int)nw[f][0];
    };
    // Where stage s has landed in this wave: its scale rows go to LDS too.
    auto publish_scales = [&](int s) {
        if constexpr (REGS) {
            const int t = tid < BM + BN ? tid : BM + BN - 1;
            *reinterpret_cast<uint2 *>(sscale + (s & 1) * ((BM + BN) * 8) + t * 8) = rs;
        }
    };
    constexpr std::integral_constant<int, 0> q0;
    constexpr std::integral_constant<int, 1> q1;
    constexpr std::integral_constant<int, 2> q2;
    constexpr std::integral_constant<int, 3> q3;
    constexpr int RQ = FM * XH + FN, MQ = FM * FN * kParts<XF>;

    if constexpr (!REGS) issue_scales(0);
    issue(0);
    publish_scales(0);  // (waits for its row; the ring is empty anyway)
#pragma unroll
    for (int s = 1; s < STA; ++s)
        if (s < nk) issue(s);
    wait_stages<STA - 1, L + (REGS ? 1 : 0)>((nk < STA ? nk : STA) - 1);  // stage 0 landed
    lds_barrier();
    // (Fragments are read one quarter before they multiply; two quarters, with
    // four sets of registers, measured no faster at any shape.)
    XFrag<XF> xa[FM], xb[FM];
    int4v wa[FN], wb[FN];
    read_scales(0);
    read_frags(0, 0, xa, wa);
    // A stage: its last quarter multiplies behind the barrier, while the next
    // stage's first fragments are read and stage kt + STA's loads issue.  The
    // empty asm keeps the sums of the first three quarters before the barrier:
    // their next use is behind a branch (the scales), and the compiler would
    // move all of their multiplies there, past every wait (measured: the matrix
    // cores 26 % busy).  The scale area is refilled in the first of its CH
    // stages, when every wave has read it.
    auto stage = [&](int kt, auto issue_c) __attribute__((always_inline)) {
        constexpr bool ISSUE = decltype(issue_c)::value;
        take_scales();
        read_frags(kt, 1, xb, wb);
        mma(q0, xa, wa);
        mx_sched<MQ, RQ, 0>();
        read_frags(kt, 2, xa, wa);
        mma(q1, xb, wb);
        mx_sched<MQ, RQ, 0>();
        read_frags(kt, 3, xb, wb);
        mma(q2, xa, wa);
        mx_sched<MQ, RQ, 0>();
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) asm volatile("" : "+v"(acc[i][j]));
        if constexpr (ISSUE) wait_vmcnt<(STA - 2) * L>();  // stage kt + 1 landed
        else wait_stages<STA - 2, L>(nk - kt - 2);
        publish_scales(kt + 1);
        lds_barrier();  // every wave has read stage kt: its slot is free
        read_scales(kt + 1);
        if constexpr (!REGS)
            if ((kt & (SN - 1)) == 0 && kt + SN < nk) issue_scales(kt / SN + 1);
        read_frags(kt + 1, 0, xa, wa);
        if constexpr (ISSUE) issue(kt + STA);
        mma(q3, xb, wb);
        mx_sched<MQ, RQ, ISSUE ? L : 0>();
    };
    int kt = 0;
    for (; kt + STA < nk; ++kt) stage(kt, std::true_type{});
    for (; kt + 1 < nk; ++kt) stage(kt, std::false_type{});  // nothing left to issue
    {  // the last stage: the weights of blocks that are added already are zero
        auto masked = [&](int q, int4v (&wf)[FN]) __attribute__((always_inline)) {
#pragma unroll
            for (int f = 0; f < FN; ++f) wf[f] = 4 * fh + q >= skip ? wf[f] : int4v{0, 0, 0, 0};
        };
        take_scales();
        read_frags(kt, 1, xb, wb);
        masked(0, wa);
        mma(q0, xa, wa);
        read_frags(kt, 2, xa, wa);
        masked(1, wb);
        mma(q1, xb, wb);
        read_frags(kt, 3, xb, wb);
        masked(2, wa);
        mma(q2, xa, wa);
        masked(3, wb);
        mma(q3, xb, wb);
    }
    wait_vmcnt<0>();
    __syncthreads();  // the ring becomes the output slabs
    if (p.y_dt == F32) mx_epilogue<BM, BN, WM, WN, F32>(p, acc, smem, m0, n0);
    else if (p.y_dt == F16) mx_epilogue<BM, BN, WM, WN, F16>(p, acc, smem, m0, n0);
    else mx_epilogue<BM, BN, WM, WN, BF16>(p, acc, smem, m0, n0);
}

// ---------------------------------------------------------------- decode

// M <= 32, or K < 256 in slabs of 32 tokens (tiles_n blocks a slab).  Bound by
// the weight stream, so a block of NW waves (eight, for K < 256 as many as it has
// windows) reads each byte of its weight rows once and everything else is kept
// small: the waves split K, each holds its part of the 16 FT activation rows for
// all of the block's weight rows, and streams its part of these, a group of 16
// rows at a time, through a private ring of S LDS stages by direct-to-LDS loads.
// No barrier until the end, where the waves' sums are added through LDS in wave
// order.
//
// A stage is a window of 128 SPW elements (64 SPW bytes) of a group's rows.
// Wave w has windows w, w + NW, ..., and holds the activations of WPW of them at
// a time: the eight waves read successive bytes of a row together (with two
// neighbouring windows a wave instead, the waves in step read every other
// 256 bytes: 27 us against 23 at M = 1, N = 28672, K = 8192).  Which blocks of a
// window meet in an instruction is free as long as both operands agree: lane
// group g takes the SPW successive blocks SPW g + j in steps j, so its scale
// bytes are SPW successive bytes of the row (one load, byte j selected by the
// instruction), and the 16-byte e4m3 chunks are those that the instruction
// pairs with these blocks (the file comment).
//
// Measured there: M = 1 22.6 us (5.5 TB/s with the launch, of the 7.0 that a
// read of this size reaches: the rest is the ring's first fill and the join at
// the end), M = 32 26.1 us with e2m1 and 31.6 with e4m3 activations.
//
// Blocks past K: their activation chunks are zero and their scales 1; the
// weight lanes re-read the row's first chunk (e2m1 codes are all finite).
template <int SPW>
__device__ __forceinline__ int dec_chunk_swz(int r) {
    // rows of 4 SPW chunks; the 16 rows a quarter-wave reads fall in distinct
    // 16-byte slots of a 256-byte bank window
    return SPW >= 4 ? r : SPW == 2 ? (r >> 1) & 7 : (r >> 2) & 3;
}

// SPW successive scale bytes from byte b of a row of KB, 127 past its end, in
// the low bytes.
template <int SPW>
__device__ __forceinline__ uint32_t dec_scales(const uint8_t *row, int b, int KB) {
    uint32_t s = 0x7f7f7f7fu;
    if (b + SPW <= KB) {
        __builtin_memcpy(&s, row + b, SPW);
    } else {
#pragma unroll
        for (int j = 0; j < SPW; ++j)
            if (b + j < KB) s = (s & ~(0xffu << (8 * j))) | ((uint32_t)row[b + j] << (8 * j));
    }
    return s;
}

// Where a wave's sums of a fragment lie in LDS for the join: lane (ri, rg)'s
// four (one token, four successive weight rows) at 16-byte slot
// 16 rg + (ri ^ (4 rg + group)), so that both the lanes that write and the
// threads that read successive rows of a token spread over the banks.
__device__ __forceinline__ int join_slot(int ri, int rg, int group) {
    return 16 * rg + (ri ^ ((4 * rg + group) & 15));
}

// The sums of the NW waves in wave order, four successive outputs a thread.
template <int YDT, int FT, int NG, int NW>
__device__ __forceinline__ void dec_store(const MxArgs &p, const f32x4 *red, int64_t ms, int M,
                                          int n0) {
    using T = typename OutT<YDT>::T;
    const int N = p.N, quads = p.groups * 4;
    const bool vec_y = N % 4 == 0 && ((uintptr_t)p.y % (4 * sizeof(T))) == 0;
    for (int e = threadIdx.x; e < quads * M; e += 64 * NW) {
        const int nq = e % quads, m = e / quads;
        const int g = nq >> 2, n = n0 + nq * 4;
        if (n >= N) continue;
        const f32x4 *r = red + (g * FT + (m >> 4)) * 64 + join_slot(m & 15, nq & 3, g);
        f32x4 s = r[0];
#pragma unroll
        for (int w = 1; w < NW; ++w) s += r[w * (NG * FT * 64)];
        T h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = narrow<YDT>(s[k]);
        T *yp = reinterpret_cast<T *>(p.y) + (ms + m) * N + n;
        if (vec_y) {  // N % 4 == 0: all four or none
            if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4 *>(yp) = __builtin_bit_cast(uint4, h);
            else *reinterpret_cast<uint2 *>(yp) = __builtin_bit_cast(uint2, h);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (n + k < N) yp[k] = h[k];
        }
    }
}

template <int XF, int FT, int SPW, int WPW, int NG, int S, int NW>
__global__ __launch_bounds__(64 * NW, 1) void mx_gemm_dec(MxArgs p) {
    constexpr int XH = XF == E4M3 ? 2 : 1;
    constexpr int SLOT = SPW * 1024;          // one stage: 16 rows of 64 SPW bytes
    constexpr int RING = S * SLOT;
    constexpr int RED = NG * FT * 1024;       // one wave's sums
    constexpr int LDSB = NW * (RING > RED ? RING : RED);
    constexpr int CPR = 4 * SPW;              // 16-byte chunks per row and stage
    constexpr int RPI = 64 / CPR;             // rows per 1 KB load
    constexpr int WB = 4 * SPW;               // blocks per window
    static_assert(SPW == 1 || SPW == 2 || SPW == 4, "one scale word per window");
    static_assert(S >= 2 && S * SPW < 64 && LDSB <= 160 * 1024, "ring");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[LDSB];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int N = p.N, K = p.K, KB = K >> 5;
    const int64_t ms = (int64_t)(blockIdx.x / p.tiles_n) * (16 * FT);  // the slab's first token
    const int M = p.M - ms < 16 * FT ? (int)(p.M - ms) : 16 * FT;
    const int ng = p.groups;
    const int n0 = (blockIdx.x % p.tiles_n) * ng * 16;
    const int ri = lane & 15, rg = lane >> 4;  // operand row and lane group
    const uint8_t *xs = p.xs + ms * KB, *xq = p.xq + ms * KB * (16 * XH);
    // this wave's windows: wave, wave + 8, ..., WPW of them a pass (those past
    // K are all zero)
    const int nwin = (KB + WB - 1) / WB;
    const int passes = nwin > wave ? (nwin - wave + NW * WPW - 1) / (NW * WPW) : 0;

    // Loader: in load i lane l fetches row i RPI + l / CPR of the group, chunk
    // (l % CPR) ^ f(row) of the window.
    const uint32_t ring = (uint32_t)(uintptr_t)(lds_void_t *)smem + (uint32_t)(wave * RING);
    const int lrow = lane / CPR, lpos = lane % CPR;
    const int ntop = N - 1 - n0;
    const uint8_t *wq0 = p.wq + (int64_t)n0 * KB * 16;
    int iw = 0, ig = 0, ip = 0, islot = 0;  // window, group, pass and slot of the next issue
    auto issue = [&]() {
        const int b0 = ((ip * WPW + iw) * NW + wave) * WB;
        uint32_t off[SPW];
#pragma unroll
        for (int i = 0; i < SPW; ++i) {
            const int r = ig * 16 + i * RPI + lrow;
            const int c = b0 + (lpos ^ dec_chunk_swz<SPW>((i * RPI + lrow) & 15));
            off[i] = ((uint32_t)(r < ntop ? r : ntop) * (uint32_t)KB + (c < KB ? c : 0)) * 16u +
                     dma_bias<16>(i);
        }
        lds_dma_based<SPW, 16, true>(off, wq0, ring + (uint32_t)(islot * SLOT));
        islot = islot + 1 == S ? 0 : islot + 1;
        if (++iw == WPW) {
            iw = 0;
            if (++ig == ng) {
                ig = 0;
                ++ip;
            }
        }
    };
    // Activations.  Up to 16 rows: each lane loads its own chunks (few lines
    // an instruction where rows repeat or are few).  More rows (XRING): such
    // loads would look up 64 lines each (27.3 us against 26.0 at M = 32,
    // N = 28672, K = 8192), so the rows come through the ring, XST stages before
    // a pass's weights: 16 rows of a window's 64 SPW bytes, or of one of its
    // halves (e4m3).
    constexpr bool XRING = FT > 1;
    constexpr int XST = XRING ? FT * WPW * XH : 0;
    int ix = 0;  // activation stages of the pass issued
    auto issue_x = [&]() {
        const int f = ix / (WPW * XH), v = ix / XH % WPW, hh = ix % XH;
        const int c0 = ((ip * WPW + v) * NW + wave) * (WB * XH) + hh * CPR;  // the stage's first chunk
        uint32_t off[SPW];
#pragma unroll
        for (int i = 0; i < SPW; ++i) {
            const int r = i * RPI + lrow;
            const int m = f * 16 + r < M ? f * 16 + r : M - 1;
            const int c = c0 + (lpos ^ dec_chunk_swz<SPW>(r));
            off[i] = ((uint32_t)m * (uint32_t)(KB * XH) + (c < KB * XH ? c : 0)) * 16u + dma_bias<16>(i);
        }
        lds_dma_based<SPW, 16, false>(off, xq, ring + (uint32_t)(islot * SLOT));
        islot = islot + 1 == S ? 0 : islot + 1;
        ++ix;
    };
    auto issue_next = [&]() {
        if (XRING && ix < XST) {
            issue_x();
        } else {
            issue();
            if (XRING && iw == 0 && ig == 0) ix = 0;  // the next pass
        }
    };
    const int nst = passes * (ng * WPW + XST);
#pragma unroll
    for (int t = 0; t < S - 1; ++t)
        if (t < nst) issue_next();

    f32x4 acc[NG][FT];
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int t = 0; t < FT; ++t) acc[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const uint8_t *rd = smem + wave * RING + ri * (64 * SPW);
    const int fsw = dec_chunk_swz<SPW>(ri);

    int t = 0, slot = 0;
    // Wait for stage t, refill the ring, and the address of the stage's row of
    // this lane.
    auto next_stage = [&]() {
        // Stage t has landed once at most min(S - 2, nst - 1 - t) later ones
        // are in flight (loads complete in order).
        wait_stages<S - 2, SPW>(nst - 1 - t);
        asm volatile("" ::: "memory");  // no read of the stage moves above the wait
        if (t + S - 1 < nst) {
            // the slot of stage t - 1 is refilled: its reads must be done
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            issue_next();
        }
        const uint8_t *sb = rd + slot * SLOT;
        ++t;
        slot = slot + 1 == S ? 0 : slot + 1;
        return sb;
    };
    for (int pass = 0; pass < passes; ++pass) {
        // this pass's activations and every group's weight scales
        XFrag<XF> xf[FT][WPW][SPW][kParts<XF>];  // (split once here, for every group)
        uint32_t sx[FT][WPW], sw[NG][WPW];
#pragma unroll
        for (int f = 0; f < FT; ++f) {
            const int m = f * 16 + ri < M ? f * 16 + ri : M - 1;
            const uint8_t *row = xq + (int64_t)m * KB * (16 * XH);
#pragma unroll
            for (int v = 0; v < WPW; ++v) {
                const int bw = ((pass * WPW + v) * NW + wave) * WB;
                sx[f][v] = dec_scales<SPW>(xs + (int64_t)m * KB, bw + SPW * rg, KB);
                if constexpr (XRING) continue;
#pragma unroll
                for (int j = 0; j < SPW; ++j) {
                    XFrag<XF> x;
#pragma unroll
                    for (int c = 0; c < XH; ++c) {
                        const int b = XF == E4M3 ? bw + SPW * (2 * c + (rg >> 1)) + j : bw + SPW * rg + j;
                        const int off = XF == E4M3 ? 32 * b + 16 * (rg & 1) : 16 * b;
                        const int4v q = *reinterpret_cast<const int4v *>(row + (b < KB ? off : 0));
                        x.c[c] = b < KB ? q : int4v{0, 0, 0, 0};
                    }
                    set_parts(xf[f][v][j], x);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            const int n = i * 16 + ri < ntop ? i * 16 + ri : ntop;
            const uint8_t *row = p.ws + (int64_t)(n0 + n) * KB;
#pragma unroll
            for (int v = 0; v < WPW; ++v)
                sw[i][v] = dec_scales<SPW>(row, ((pass * WPW + v) * NW + wave) * WB + SPW * rg, KB);
        }
        if constexpr (XRING) {
            // (the scale words are taken before the first stage: a wait for
            // them later would wait for the whole ring)
#pragma unroll
            for (int v = 0; v < WPW; ++v) {
#pragma unroll
                for (int f = 0; f < FT; ++f) asm volatile("" : "+v"(sx[f][v]));
#pragma unroll
                for (int i = 0; i < NG; ++i) asm volatile("" : "+v"(sw[i][v]));
            }
#pragma unroll
            for (int f = 0; f < FT; ++f)
#pragma unroll
                for (int v = 0; v < WPW; ++v) {
                    XFrag<XF> x[SPW];
#pragma unroll
                    for (int c = 0; c < XH; ++c) {
                        const uint8_t *sb = next_stage();
                        const int bw = ((pass * WPW + v) * NW + wave) * WB;
#pragma unroll
                        for (int j = 0; j < SPW; ++j) {
                            const int b = XF == E4M3 ? bw + SPW * (2 * c + (rg >> 1)) + j : bw + SPW * rg + j;
                            const int ch = XF == E4M3 ? 2 * (SPW * (rg >> 1) + j) + (rg & 1) : SPW * rg + j;
                            const int4v q = *reinterpret_cast<const int4v *>(sb + ((ch ^ fsw) << 4));
                            x[j].c[c] = b < KB ? q : int4v{0, 0, 0, 0};
                        }
                    }
#pragma unroll
                    for (int j = 0; j < SPW; ++j) set_parts(xf[f][v][j], x[j]);
                }
        }
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            if (i < ng) {
#pragma unroll
                for (int v = 0; v < WPW; ++v) {
                    const uint8_t *sb = next_stage();
                    int4v wf[SPW];
#pragma unroll
                    for (int j = 0; j < SPW; ++j)
                        wf[j] = *reinterpret_cast<const int4v *>(sb + (((SPW * rg + j) ^ fsw) << 4));
                    auto step = [&](auto jc) {
                        constexpr int J = decltype(jc)::value;
                        if constexpr (J < SPW) {
#pragma unroll
                            for (int h = 0; h < kParts<XF>; ++h)
#pragma unroll
                                for (int f = 0; f < FT; ++f)
                                    acc[i][f] = mfma16<XF, J>(wf[J], xf[f][v][J][h], acc[i][f],
                                                              (int)sw[i][v], (int)sx[f][v]);
                        }
                    };
                    step(std::integral_constant<int, 0>{});
                    step(std::integral_constant<int, 1>{});
                    step(std::integral_constant<int, 2>{});
                    step(std::integral_constant<int, 3>{});
                }
            }
        }
    }
    wait_vmcnt<0>();
    __syncthreads();  // every wave is done with its ring: reuse it for the sums

    // 16x16 accumulator layout: lane l, register v holds weight row
    // 4 (l / 16) + v and token l % 16.
    f32x4 *red = reinterpret_cast<f32x4 *>(smem);  // [wave][group][f][slot]
#pragma unroll
    for (int i = 0; i < NG; ++i)
        if (i < ng) {
#pragma unroll
            for (int f = 0; f < FT; ++f)
                red[((wave * NG + i) * FT + f) * 64 + join_slot(ri, rg, i)] = acc[i][f];
        }
    __syncthreads();
    if (p.y_dt == F32) dec_store<F32, FT, NG, NW>(p, red, ms, M, n0);
    else if (p.y_dt == F16) dec_store<F16, FT, NG, NW>(p, red, ms, M, n0);
    else dec_store<BF16, FT, NG, NW>(p, red, ms, M, n0);
}

// ---------------------------------------------------------------- launch

// The launchers enqueue nothing and return false where the blocks are more
// than a grid can hold (2^32 threads along one dimension).
static bool grid_holds(int64_t blocks, int threads) { return blocks * threads < (int64_t)1 << 32; }

template <int XF, int BM, int BN, int WM, int WN, int STA, int CH>
static bool launch_pp(MxArgs &a, hipStream_t stream) {
    const int tm = (a.M + BM - 1) / BM, tn = (a.N + BN - 1) / BN;
    const dim3 block(64 * WM * WN);
    if (!grid_holds((int64_t)tm * tn, (int)block.x)) return false;
    set_xcd_grid(a, tm, tn, BM, BN);
    mx_gemm_pp<XF, BM, BN, WM, WN, STA, CH><<<dim3((unsigned)(tm * tn)), block, 0, stream>>>(a);
    return true;
}

template <int XF, int FT, int SPW, int WPW, int NG, int S, int NW = 8>
static bool launch_dec_t(MxArgs &a, hipStream_t stream) {
    a.tiles_n = (a.N + 16 * a.groups - 1) / (16 * a.groups);
    const int64_t blocks = (((int64_t)a.M + 16 * FT - 1) / (16 * FT)) * a.tiles_n;
    // (one limit for one wave a block and two, the one that sq_mx.h states)
    if (!grid_holds(blocks, NW == 8 ? 512 : 128)) return false;
    mx_gemm_dec<XF, FT, SPW, WPW, NG, S, NW><<<dim3((unsigned)blocks), 64 * NW, 0, stream>>>(a);
    return true;
}

// M <= 32, K >= 256.
template <int XF, int FT>
static bool launch_dec(MxArgs &a, hipStream_t stream) {
    // groups of 16 weight rows per block: an equal share for the 256 CUs of
    // as few rounds of blocks as eight groups a block allow
    const int64_t groups = ((int64_t)a.N + 15) / 16;
    const int64_t rounds = (groups + 256 * 8 - 1) / (256 * 8);
    a.groups = (int)((groups + 256 * rounds - 1) / (256 * rounds));
    // the windows that let eight waves cover K, at most 1024 elements a wave
    // (512 where the activations of 32 rows would not fit the registers)
    constexpr int kMaxWpw = XF == E2M1 || FT == 1 ? 2 : 1;
    const bool many = a.groups > 2;
    if (a.K <= 1024) {
        return many ? launch_dec_t<XF, FT, 1, 1, 8, 8>(a, stream)
                    : launch_dec_t<XF, FT, 1, 1, 2, 3>(a, stream);
    } else if (a.K <= 2048) {
        return many ? launch_dec_t<XF, FT, 2, 1, 8, 6>(a, stream)
                    : launch_dec_t<XF, FT, 2, 1, 2, 3>(a, stream);
    } else if (a.K <= 4096 || kMaxWpw == 1) {
        return many ? launch_dec_t<XF, FT, 4, 1, 8, 4>(a, stream)
                    : launch_dec_t<XF, FT, 4, 1, 2, 3>(a, stream);
    } else if constexpr (kMaxWpw == 2) {
        return many ? launch_dec_t<XF, FT, 4, 2, 8, 4>(a, stream)
                    : launch_dec_t<XF, FT, 4, 2, 2, 4>(a, stream);
    }
}

// K < 256: slabs of 16 FT tokens, as many waves a block as K has windows of 128
// elements (NW), and two groups of weight rows a block, one where that leaves
// fewer than four blocks a CU.  us, fp16 outputs:
//   groups            4096 x 4096 x 64   x 224   1693 x 11440 x 64   64 x 4096 x 128
//   e2m1  1                31.4          43.6          42.7                3.3
//         2                19.1          26.2          27.6                3.7
//         4                26.4          44.9          34.5                6.1
//         8                21.3          35.9          28.2                8.2
//         launch_dec's     81.5          90.6         172.2                3.5
//   e4m3  1                38.2          58.6          49.6                3.8
//         2                23.3          34.8          32.9                4.1
//         8                22.9          39.6          30.8                8.9
// and of few tokens, launch_dec's against these: 8 x 70000 x 64 10.0 and 4.0,
// 32 x 28672 x 224 8.2 and 5.1, 1 x 4096 x 64 2.7 and 2.5.  (fp32 outputs of
// 4096 x 4096 x 64 20.5; filling them alone takes 12.)
template <int XF, int FT, int NW>
static bool launch_short(MxArgs &a, hipStream_t stream) {
    const int64_t blocks = (((int64_t)a.M + 16 * FT - 1) / (16 * FT)) * (((int64_t)a.N + 15) / 16);
    a.groups = blocks > 1024 && a.N > 16 ? 2 : 1;
    return launch_dec_t<XF, FT, 1, 1, 2, 3, NW>(a, stream);
}

template <int XF>
static bool launch_mx(MxArgs &a, hipStream_t stream, int tile) {
    if (a.K <= 128) return a.M <= 16 ? launch_short<XF, 1, 1>(a, stream) : launch_short<XF, 2, 1>(a, stream);
    if (a.K < 256) return a.M <= 16 ? launch_short<XF, 1, 2>(a, stream) : launch_short<XF, 2, 2>(a, stream);
    if (a.M <= 16) return launch_dec<XF, 1>(a, stream);
    if (a.M <= 32) return launch_dec<XF, 2>(a, stream);
    if (a.K % 128 != 0) {
        if (tile == 3) return launch_pp<XF, 64, 128, 2, 4, 2, 0>(a, stream);
        // (e4m3: one m-fragment a wave, so that fewer waves split the same
        // activations; 333 x 5001 x 1056 in these tiles 13.6 us, with two 15.6;
        // 256 x 28672 x 7168 in 128 x 256 tiles 87 and 95)
        constexpr int WM = XF == E4M3 ? 4 : 2;
        return launch_pp<XF, 128, 128, WM, 8 / WM, 2, 0>(a, stream);
    }
    if constexpr (XF == E2M1) {
        if (tile == 0) return launch_pp<XF, 256, 256, 4, 2, 2, 2>(a, stream);
        if (tile == 1) return launch_pp<XF, 256, 128, 4, 2, 3, 4>(a, stream);
        if (tile == 2) return launch_pp<XF, 128, 128, 2, 2, 2, 4>(a, stream);
        return launch_pp<XF, 64, 128, 2, 4, 3, 4>(a, stream);
    } else {
        if (tile == 0) return launch_pp<XF, 128, 256, 4, 2, 2, 4>(a, stream);
        if (tile < 3) return launch_pp<XF, 128, 128, 4, 2, 3, 4>(a, stream);
        return launch_pp<XF, 64, 128, 2, 4, 3, 4>(a, stream);
    }
}

// The block tile of M > 32: the least rounds of tiles over the 256 CUs, each
// taking its outputs over the shape's rate.  The rates are relative to the
// largest shape's, from these times (us; 16-bit outputs; tiles as numbered in
// launch_mx):                         0      1      2      3
//   e2m1  4096 x 14336 x 4096        133.9  149.4  157.9  247.7
//         4096 x 4096 x 1024          16.3   17.8   16.4   22.3
//         2048 x 4096 x 4096          27.1   22.9   23.0   30.3
//         4096 x 1024 x 1024          10.9    8.5    7.2    7.4
//         256 x 28672 x 7168          60.5   41.3   41.0   60.2
//         64 x 28672 x 8192           58.0   39.8   40.9   30.6
//         256 x 4096 x 4096           25.6   17.5   16.1   11.1
//         128 x 8192 x 8192           56.0   34.2   38.3   23.2
//         33 x 1024 x 4096            23.6   16.3   15.5   10.5
//         2048 x 512 x 4096           25.4   17.6   16.0   11.0
//   e4m3  4096 x 14336 x 4096        317       -   389    543
//         4096 x 4096 x 1024          29.8     -    35.9   50.4
//         2048 x 4096 x 4096          49.3     -    59.4   80.3
//         256 x 28672 x 7168          87.4     -    97.9  136
//         256 x 4096 x 4096           39.7     -    26.0   20.3
//         128 x 28672 x 8192          81.6     -    56.6   81.8
//         33 x 1024 x 4096            37.5     -    24.5   19.1
//         333 x 5001 x 1024           16.6     -    11.9    9.0
// Over 54 shapes a format, M = 33 .. 8192 and N = 300 .. 28672, the choice was the
// fastest shape or within 8 % of it but for e2m1 with 64 x 128 tiles in two short
// rounds, which run two blocks a CU (1000 x 4096 x 4096 20.3 us, 17.6 in those;
// 8192 x 300 x 1024 10.7, 8.2).
static int mx_pick_tile(int x_fmt, int64_t M, int64_t N, int64_t K) {
    struct C { int bm, bn; double rate; };
    const C e2[4] = {{256, 256, 1.0}, {256, 128, 0.85}, {128, 128, 0.7}, {64, 128, 0.5}};
    const C e4[4] = {{128, 256, 1.0}, {128, 128, 0.7}, {128, 128, 0.7}, {64, 128, 0.5}};
    int best = 0;
    double least = 0;
    for (int i = K % 128 != 0 ? 2 : 0; i < 4; ++i) {
        const C &c = x_fmt == E2M1 ? e2[i] : e4[i];
        const int64_t tiles = ((M + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn);
        const double t = (double)((tiles + 255) / 256) * c.bm * c.bn / c.rate;
        if (least == 0 || t < least * 0.999) { least = t; best = i; }
    }
    return best;
}

bool launch_gemm_mx(const uint8_t *xq, const uint8_t *xs, int x_fmt, const uint8_t *wq,
                    const uint8_t *ws, int64_t M, int64_t N, int64_t K, void *y, int y_dt,
                    hipStream_t stream, int force_tile) {
    MxArgs a{};
    a.xq = xq; a.xs = xs; a.wq = wq; a.ws = ws;
    a.M = (int)M; a.N = (int)N; a.K = (int)K; a.y = y; a.y_dt = y_dt;
    const int tile = force_tile >= 0 ? force_tile : mx_pick_tile(x_fmt, M, N, K);
    return x_fmt == E2M1 ? launch_mx<E2M1>(a, stream, tile) : launch_mx<E4M3>(a, stream, tile);
}

}  // namespace sq
