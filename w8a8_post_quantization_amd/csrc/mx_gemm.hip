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
// Three kernels:
//  * mx_gemm_dec   M <= 32 (decode), bound by the weight stream.
//  * mx_gemm_pp    M > 32, K % 128 == 0, K >= 256: both operands through LDS rings
//                  filled by direct-to-LDS loads.
//  * mx_gemm_tile  M > 32, other K: staged through registers.
#include <type_traits>

#include "mx_device.h"
#include "pipe_device.h"
#include "sq_launch.h"

namespace sq {

struct MxArgs : TileGrid {
    const uint8_t *xq, *xs, *wq, *ws;
    int M, N, K;
    void *y;
    int groups;  // mx_gemm_dec: groups of 16 weight rows a block covers
};

template <int YDT>
__device__ __forceinline__ void mx_store_y(void *y, int64_t i, float v) {
    reinterpret_cast<typename OutT<YDT>::T *>(y)[i] = narrow<YDT>(v);
}

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

// The four scale bytes that lane half fh needs for the four 64-element
// quarters of a stage (blocks 2 q + fh of the row's eight), byte q for
// quarter q.
__device__ __forceinline__ int quarter_scales(uint2 s, int fh) {
    return (int)__builtin_amdgcn_perm(s.y, s.x, fh ? 0x07050301u : 0x06040200u);
}

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
    const bool vec_y = ((N * (int)sizeof(T)) & 15) == 0 && ((uintptr_t)p.y & 15) == 0;
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
            if (vec_y && n + EPC <= N) {
                *reinterpret_cast<uint4 *>(yp) = v;
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

// K % 128 == 0, K >= 256.  A stage is 256 elements of K: 128 bytes of every weight row,
// 128 (e2m1) or twice 128 (e4m3, two half tiles) of every activation row, and
// the rows' eight scale bytes, streamed into a ring of STA LDS stages by
// direct-to-LDS loads.  Data rows are 128 bytes with chunk c of row r at slot
// c ^ swz(r).  A stage is consumed as four quarters of 64 elements with
// ping-pong fragment registers; the scale bytes of a row become one register
// per fragment and stage, whose byte q the instruction selects in quarter q.
// Where K % 256 == 128 the last stage is the row's last 256 elements again,
// of which the first two quarters (added already) are skipped.
template <int XF, int BM, int BN, int WM, int WN, int STA, int YDT>
__global__ __launch_bounds__(64 * WM * WN, 1) void mx_gemm_pp(MxArgs p) {
    constexpr int NW = WM * WN, XH = XF == E4M3 ? 2 : 1;
    constexpr int WTM = BM / WM, WTN = BN / WN;
    constexpr int FM = WTM / 32, FN = WTN / 32;
    constexpr int LX = BM * XH / (8 * NW), LW = BN / (8 * NW);  // 1 KB loads per wave and stage
    constexpr int LS = (BM + BN + 32 * NW - 1) / (32 * NW);     // 256 B scale loads
    constexpr int L = LX + LW + LS;
    constexpr int SX = BM * 128 * XH, SW = BN * 128, SS = LS * NW * 256;
    constexpr int STG = SX + SW + SS;
    static_assert(FM >= 1 && FN >= 1 && LX >= 1 && LW >= 1 && LS >= 1 && LS <= 4, "tile");
    static_assert(STA >= 2 && STA * L < 64, "vmcnt range");
    static_assert(NW * 32 * WTN * (int)sizeof(typename OutT<YDT>::T) <= STA * STG, "slabs");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[STA * STG];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave / WN, wn = wave % WN;
    int tile_m, tile_n;
    tile_of(p, blockIdx.x, tile_m, tile_n);
    const int m0 = tile_m * BM, n0 = tile_n * BN;
    const int M = p.M, N = p.N, K = p.K;
    const int KB = K >> 5;
    const int nk = (K + 255) >> 8;
    const bool half = (K & 128) != 0;  // the last stage adds 128 elements

    // This wave's loads: offsets of its lanes from the tile's first row (rows
    // past the edge read a valid row, whose outputs are never stored).
    uint32_t x_off[LX], w_off[LW], s_off[LS];
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
    // Scale rows: the tile's activation rows (load instructions below LSX of
    // the block's LS NW), then its weight rows; those past both repeat the last.
    constexpr int LSX = BM / 32;
    const uint8_t *xs0 = p.xs + (int64_t)m0 * KB, *ws0 = p.ws + (int64_t)n0 * KB;
#pragma unroll
    for (int j = 0; j < LS; ++j) {
        const int i = wave * LS + j;
        int row = (i < LSX ? i : i - LSX) * 32 + (lane >> 1);
        const int top = i < LSX ? mtop : ntop < BN - 1 ? ntop : BN - 1;
        row = row < top ? row : top;
        s_off[j] = (uint32_t)row * (uint32_t)KB + 4 * (lane & 1) + dma_bias<4>(0);
    }
    const uint32_t waveu = (uint32_t)__builtin_amdgcn_readfirstlane(wave);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void_t *)smem;
    const uint8_t *xq0 = p.xq + (int64_t)m0 * (K * (int64_t)XH / 2), *wq0 = p.wq + (int64_t)n0 * (K / 2);
    auto issue = [&](int s) {  // stage s < nk
        const uint32_t base = lds0 + (uint32_t)((s % STA) * STG);
        const int b0 = s * 8 < KB - 8 ? s * 8 : KB - 8;  // the stage's first block
        lds_dma_based<LX, 16, false>(x_off, xq0 + b0 * (16 * XH), base + waveu * (LX * 1024u));
        lds_dma_based<LW, 16, false>(w_off, wq0 + b0 * 16, base + SX + waveu * (LW * 1024u));
#pragma unroll
        for (int j = 0; j < LS; ++j)
            lds_dma_based<1, 4, false>(s_off + j, ((int)(waveu * LS) + j < LSX ? xs0 : ws0) + b0,
                                       base + SX + SW + (waveu * LS + j) * 256u);
    };

    const int fr = lane & 31, fh = lane >> 5;
    const int fsw = swz(fr);  // fragment bases are multiples of 32 rows
    auto read_frags = [&](int s, int q, XFrag<XF> (&xf)[FM], int4v (&wf)[FN]) {
        const uint8_t *xb = smem + (s % STA) * STG + (XF == E4M3 ? (q >> 1) * (BM * 128) : 0);
        const uint8_t *wb = smem + (s % STA) * STG + SX;
#pragma unroll
        for (int f = 0; f < FM; ++f)
#pragma unroll
            for (int c = 0; c < XH; ++c) {
                const int ch = XF == E4M3 ? 4 * (q & 1) + 2 * c + fh : 2 * q + fh;
                xf[f].c[c] = *reinterpret_cast<const int4v *>(
                    xb + (wm * WTM + f * 32 + fr) * 128 + ((ch ^ fsw) << 4));
            }
#pragma unroll
        for (int f = 0; f < FN; ++f)
            wf[f] = *reinterpret_cast<const int4v *>(wb + (wn * WTN + f * 32 + fr) * 128 +
                                                     (((2 * q + fh) ^ fsw) << 4));
    };
    auto read_scales = [&](int s, uint2 (&sx)[FM], uint2 (&sw)[FN]) {
        const uint2 *sb = reinterpret_cast<const uint2 *>(smem + (s % STA) * STG + SX + SW);
#pragma unroll
        for (int f = 0; f < FM; ++f) sx[f] = sb[wm * WTM + f * 32 + fr];
#pragma unroll
        for (int f = 0; f < FN; ++f) sw[f] = sb[BM + wn * WTN + f * 32 + fr];
    };

    f32x16 acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    int cx[FM], cw[FN];  // this stage's scales
    auto mma = [&](auto qc, const XFrag<XF> (&xf)[FM], const int4v (&wf)[FN]) {
        constexpr int Q = decltype(qc)::value;
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j)
                acc[i][j] = mfma32<XF, Q>(wf[i], xf[j], acc[i][j], cw[i], cx[j]);
    };
    auto take_scales = [&](const uint2 (&sx)[FM], const uint2 (&sw)[FN]) {
#pragma unroll
        for (int f = 0; f < FM; ++f) cx[f] = quarter_scales(sx[f], fh);
#pragma unroll
        for (int f = 0; f < FN; ++f) cw[f] = quarter_scales(sw[f], fh);
    };
    constexpr std::integral_constant<int, 0> q0;
    constexpr std::integral_constant<int, 1> q1;
    constexpr std::integral_constant<int, 2> q2;
    constexpr std::integral_constant<int, 3> q3;
    constexpr int RQ = FM * XH + FN, MQ = FM * FN;

#pragma unroll
    for (int s = 0; s < STA; ++s)
        if (s < nk) issue(s);
    wait_stages<STA - 1, L>((nk < STA ? nk : STA) - 1);  // stage 0 landed
    lds_barrier();
    XFrag<XF> xa[FM], xb[FM];
    int4v wa[FN], wb[FN];
    uint2 nx[FM], nw[FN];
    read_scales(0, nx, nw);
    read_frags(0, 0, xa, wa);
    int kt = 0;
    for (; kt + STA < nk; ++kt) {
        take_scales(nx, nw);
        read_frags(kt, 1, xb, wb);
        mma(q0, xa, wa);
        mx_sched<MQ, RQ, 0>();
        read_frags(kt, 2, xa, wa);
        mma(q1, xb, wb);
        mx_sched<MQ, RQ, 0>();
        read_frags(kt, 3, xb, wb);
        mma(q2, xa, wa);
        mx_sched<MQ, RQ, 0>();
        wait_vmcnt<(STA - 2) * L>();  // stage kt + 1 landed
        lds_barrier();                // every wave has read stage kt: its slot is free
        read_scales(kt + 1, nx, nw);
        read_frags(kt + 1, 0, xa, wa);
        issue(kt + STA);
        mma(q3, xb, wb);
        mx_sched<MQ, RQ + FM + FN, L>();
    }
    const int nfull = half ? nk - 1 : nk;
    for (; kt < nfull; ++kt) {  // nothing left to issue
        take_scales(nx, nw);
        read_frags(kt, 1, xb, wb);
        mma(q0, xa, wa);
        mx_sched<MQ, RQ, 0>();
        read_frags(kt, 2, xa, wa);
        mma(q1, xb, wb);
        mx_sched<MQ, RQ, 0>();
        read_frags(kt, 3, xb, wb);
        mma(q2, xa, wa);
        mx_sched<MQ, RQ, 0>();
        wait_stages<STA - 2, L>(nk - kt - 2);  // stage kt + 1 landed (if any)
        lds_barrier();
        read_scales(kt + 1, nx, nw);  // past the last stage: never used
        read_frags(kt + 1, 0, xa, wa);
        mma(q3, xb, wb);
    }
    if (half) {
        take_scales(nx, nw);
        read_frags(kt, 2, xa, wa);
        read_frags(kt, 3, xb, wb);
        mma(q2, xa, wa);
        mma(q3, xb, wb);
    }
    wait_vmcnt<0>();
    __syncthreads();  // the ring becomes the output slabs
    mx_epilogue<BM, BN, WM, WN, YDT>(p, acc, smem, m0, n0);
}

// Any K (a multiple of 32): 128 x 128 tiles of four waves, a stage of 256
// elements of K loaded into registers while the previous one multiplies, then
// written to one of two LDS buffers in mx_gemm_pp's layout.  Chunks past K
// are zero with scale 1.  (Scale rows of K / 32 bytes start at any byte here,
// which direct-to-LDS loads cannot fetch.)
template <int XF, int YDT>
__global__ __launch_bounds__(256, 1) void mx_gemm_tile(MxArgs p) {
    constexpr int BM = 128, BN = 128, WM = 2, WN = 2, XH = XF == E4M3 ? 2 : 1;
    constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / 32, FN = WTN / 32;
    constexpr int TX = BM * 8 * XH / 256, TW = BN * 8 / 256;  // chunks per thread and stage
    constexpr int SX = BM * 128 * XH, SW = BN * 128, SS = (BM + BN) * 8, STG = SX + SW + SS;
    static_assert(BM + BN == 256, "one scale row per thread");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * STG];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave / WN, wn = wave % WN;
    int tile_m, tile_n;
    tile_of(p, blockIdx.x, tile_m, tile_n);
    const int m0 = tile_m * BM, n0 = tile_n * BN;
    const int M = p.M, N = p.N, K = p.K, KB = K >> 5;
    const int nk = (K + 255) >> 8;

    const uint8_t *x_src[TX], *w_src[TW], *s_src;
    int x_chunk[TX], w_chunk[TW], x_lds[TX], w_lds[TW];
#pragma unroll
    for (int j = 0; j < TX; ++j) {
        const int i = tid + 256 * j, hh = i / (BM * 8), row = (i / 8) % BM, c = i & 7;
        const int64_t m = m0 + row < M ? m0 + row : M - 1;
        x_chunk[j] = hh * 8 + c;
        x_src[j] = p.xq + m * KB * (16 * XH) + x_chunk[j] * 16;
        x_lds[j] = hh * (BM * 128) + row * 128 + ((c ^ swz(row)) << 4);
    }
#pragma unroll
    for (int j = 0; j < TW; ++j) {
        const int i = tid + 256 * j, row = i / 8, c = i & 7;
        const int64_t n = n0 + row < N ? n0 + row : N - 1;
        w_chunk[j] = c;
        w_src[j] = p.wq + n * KB * 16 + c * 16;
        w_lds[j] = SX + row * 128 + ((c ^ swz(row)) << 4);
    }
    {
        const int64_t m = m0 + tid < M ? m0 + tid : M - 1;
        const int64_t n = n0 + tid - BM < N ? n0 + tid - BM : N - 1;
        s_src = tid < BM ? p.xs + m * KB : p.ws + n * KB;
    }
    uint4 rx[TX], rw[TW];
    uint2 rs;
    // (chunks past K load the row's first chunk and are zeroed after: a load
    // under a lane-dependent condition would wait for the earlier ones)
    auto load = [&](int s) {
#pragma unroll
        for (int j = 0; j < TX; ++j) {
            const bool in = s * 8 * XH + x_chunk[j] < KB * XH;
            const uint4 v = *reinterpret_cast<const uint4 *>(
                x_src[j] + (in ? s * 128 * XH : -16 * x_chunk[j]));
            rx[j] = in ? v : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < TW; ++j) {
            const bool in = s * 8 + w_chunk[j] < KB;
            const uint4 v =
                *reinterpret_cast<const uint4 *>(w_src[j] + (in ? s * 128 : -16 * w_chunk[j]));
            rw[j] = in ? v : make_uint4(0, 0, 0, 0);
        }
        if (s * 8 + 8 <= KB) {
            __builtin_memcpy(&rs, s_src + s * 8, 8);
        } else {
            uint8_t b[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint8_t v = s_src[s * 8 + i < KB ? s * 8 + i : 0];
                b[i] = s * 8 + i < KB ? v : 127;
            }
            __builtin_memcpy(&rs, b, 8);
        }
    };
    auto store = [&](int buf) {
        uint8_t *base = smem + buf * STG;
#pragma unroll
        for (int j = 0; j < TX; ++j) *reinterpret_cast<uint4 *>(base + x_lds[j]) = rx[j];
#pragma unroll
        for (int j = 0; j < TW; ++j) *reinterpret_cast<uint4 *>(base + w_lds[j]) = rw[j];
        *reinterpret_cast<uint2 *>(base + SX + SW + tid * 8) = rs;
    };

    const int fr = lane & 31, fh = lane >> 5, fsw = swz(fr);
    f32x16 acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

    load(0);
    store(0);
    __syncthreads();
    for (int kt = 0; kt < nk; ++kt) {
        if (kt + 1 < nk) load(kt + 1);
        const uint8_t *base = smem + (kt & 1) * STG;
        const uint2 *sb = reinterpret_cast<const uint2 *>(base + SX + SW);
        int cx[FM], cw[FN];
#pragma unroll
        for (int f = 0; f < FM; ++f) cx[f] = quarter_scales(sb[wm * WTM + f * 32 + fr], fh);
#pragma unroll
        for (int f = 0; f < FN; ++f) cw[f] = quarter_scales(sb[BM + wn * WTN + f * 32 + fr], fh);
        auto quarter = [&](auto qc) {
            constexpr int Q = decltype(qc)::value;
            XFrag<XF> xf[FM];
            int4v wf[FN];
#pragma unroll
            for (int f = 0; f < FM; ++f)
#pragma unroll
                for (int c = 0; c < XH; ++c) {
                    const int ch = XF == E4M3 ? 4 * (Q & 1) + 2 * c + fh : 2 * Q + fh;
                    xf[f].c[c] = *reinterpret_cast<const int4v *>(
                        base + (XF == E4M3 ? (Q >> 1) * (BM * 128) : 0) +
                        (wm * WTM + f * 32 + fr) * 128 + ((ch ^ fsw) << 4));
                }
#pragma unroll
            for (int f = 0; f < FN; ++f)
                wf[f] = *reinterpret_cast<const int4v *>(
                    base + SX + (wn * WTN + f * 32 + fr) * 128 + (((2 * Q + fh) ^ fsw) << 4));
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j)
                    acc[i][j] = mfma32<XF, Q>(wf[i], xf[j], acc[i][j], cw[i], cx[j]);
        };
        quarter(std::integral_constant<int, 0>{});
        quarter(std::integral_constant<int, 1>{});
        quarter(std::integral_constant<int, 2>{});
        quarter(std::integral_constant<int, 3>{});
        if (kt + 1 < nk) store((kt + 1) & 1);
        __syncthreads();
    }
    mx_epilogue<BM, BN, WM, WN, YDT>(p, acc, smem, m0, n0);
}

// ---------------------------------------------------------------- decode

// M <= 32.  Bound by the weight stream, so a block of eight waves reads each
// byte of its weight rows once and everything else is kept small: the waves
// split K, each holds its part of the 16 FT activation rows in registers for
// the whole kernel (read once per block), and streams its part of the weight
// rows, a group of 16 rows a stage, through a private ring of S LDS stages by
// direct-to-LDS loads.  No barrier until the end, where the waves' sums of
// every group are added through LDS in wave order.
//
// A wave's part of K is a window of 128 SPW elements (64 SPW bytes of a
// weight row); windows repeat every 8 * 128 SPW elements for a longer K.
// Which blocks of the window meet in an instruction is free as long as both
// operands agree: lane group g takes the SPW successive blocks SPW g + j in
// steps j, so its scale bytes are SPW successive bytes of the row (one load,
// byte j selected by the instruction), and the 16-byte e4m3 chunks are those
// that the instruction pairs with these blocks (the file comment).
//
// Blocks past K: their activation chunks are zero and their scales 1; the
// weight lanes re-read the row's first chunk (e2m1 codes are all finite).
template <int SPW>
__device__ __forceinline__ int dec_chunk_swz(int r) {
    // rows of 4 SPW chunks; the 16 rows a quarter-wave reads fall in distinct
    // 16-byte slots of a 256-byte bank window
    return SPW >= 4 ? r : SPW == 2 ? (r >> 1) & 7 : (r >> 2) & 3;
}

// SPW successive scale bytes from byte b of a row of KB, 127 past its end,
// byte j of word j / 4 for step j.
template <int SPW>
__device__ __forceinline__ void dec_scales(const uint8_t *row, int b, int KB, uint32_t (&s)[(SPW + 3) / 4]) {
    if (b + SPW <= KB) {
        if constexpr (SPW < 4) s[0] = 0;
        __builtin_memcpy(s, row + b, SPW);
    } else {
#pragma unroll
        for (int w = 0; w < (SPW + 3) / 4; ++w) s[w] = 0x7f7f7f7fu;
#pragma unroll
        for (int j = 0; j < SPW; ++j)
            if (b + j < KB)
                s[j / 4] = (s[j / 4] & ~(0xffu << (8 * (j & 3)))) | ((uint32_t)row[b + j] << (8 * (j & 3)));
    }
}

template <int XF, int FT, int SPW, int NG, int S, int YDT>
__global__ __launch_bounds__(512, 1) void mx_gemm_dec(MxArgs p) {
    constexpr int NW = 8, XH = XF == E4M3 ? 2 : 1;
    constexpr int SLOT = SPW * 1024;          // one stage: 16 rows of 64 SPW bytes
    constexpr int RING = S * SLOT;
    constexpr int RED = NG * FT * 1024;       // one wave's sums
    constexpr int LDSB = NW * (RING > RED ? RING : RED);
    constexpr int CPR = 4 * SPW;              // 16-byte chunks per row and stage
    constexpr int RPI = 64 / CPR;             // rows per 1 KB load
    constexpr int SWORDS = (SPW + 3) / 4;
    static_assert(RPI >= 1 && RPI * SPW == 16, "a load covers whole rows");
    static_assert(S >= 2 && S * SPW < 64 && LDSB <= 160 * 1024, "ring");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[LDSB];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int M = p.M, N = p.N, K = p.K, KB = K >> 5;
    const int ng = p.groups;
    const int n0 = blockIdx.x * ng * 16;
    const int ri = lane & 15, rg = lane >> 4;  // operand row and lane group
    constexpr int WB = 4 * SPW;                // blocks per window
    // windows of this wave: wave, wave + 8, ... below nwin
    const int nwin = (KB + WB - 1) / WB;
    const int mine = nwin > wave ? (nwin - wave + NW - 1) / NW : 0;

    // Loader: in load i lane l fetches row i RPI + l / CPR of the group, chunk
    // (l % CPR) ^ f(row) of the window.
    const uint32_t ring = (uint32_t)(uintptr_t)(lds_void_t *)smem + (uint32_t)(wave * RING);
    const int lrow = lane / CPR, lpos = lane % CPR;
    const int ntop = N - 1 - n0;
    const uint8_t *wq0 = p.wq + (int64_t)n0 * KB * 16;
    auto issue = [&](int t) {  // stage t: window wave + 8 (t / ng), group t % ng
        const int win = wave + NW * (t / ng), grp = t % ng;
        const uint32_t slot = ring + (uint32_t)((t % S) * SLOT);
        uint32_t off[SPW];
#pragma unroll
        for (int i = 0; i < SPW; ++i) {
            const int r = grp * 16 + i * RPI + lrow;
            const int c = win * WB + (lpos ^ dec_chunk_swz<SPW>((i * RPI + lrow) & 15));
            off[i] = ((uint32_t)(r < ntop ? r : ntop) * (uint32_t)KB + (c < KB ? c : 0)) * 16u +
                     dma_bias<16>(i);
        }
        lds_dma_based<SPW, 16, true>(off, wq0, slot);
    };
    const int nst = mine * ng;
#pragma unroll
    for (int t = 0; t < S - 1; ++t)
        if (t < nst) issue(t);

    f32x4 acc[NG][FT];
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int t = 0; t < FT; ++t) acc[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const uint8_t *rd = smem + wave * RING + ri * (64 * SPW);
    const int fsw = dec_chunk_swz<SPW>(ri);

    int t = 0;
    for (int w = 0; w < mine; ++w) {
        const int b0 = (wave + NW * w) * WB;  // the window's first block
        // this window's activations and every group's weight scales
        XFrag<XF> xf[FT][SPW];
        uint32_t sx[FT][SWORDS], sw[NG][SWORDS];
#pragma unroll
        for (int f = 0; f < FT; ++f) {
            const int m = f * 16 + ri < M ? f * 16 + ri : M - 1;
            dec_scales<SPW>(p.xs + (int64_t)m * KB, b0 + SPW * rg, KB, sx[f]);
            const uint8_t *row = p.xq + (int64_t)m * KB * (16 * XH);
#pragma unroll
            for (int j = 0; j < SPW; ++j)
#pragma unroll
                for (int c = 0; c < XH; ++c) {
                    const int b = XF == E4M3 ? b0 + SPW * (2 * c + (rg >> 1)) + j : b0 + SPW * rg + j;
                    const int off = XF == E4M3 ? 32 * b + 16 * (rg & 1) : 16 * b;
                    const int4v v = *reinterpret_cast<const int4v *>(row + (b < KB ? off : 0));
                    xf[f][j].c[c] = b < KB ? v : int4v{0, 0, 0, 0};
                }
        }
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            const int n = n0 + i * 16 + ri < N ? n0 + i * 16 + ri : N - 1;
            dec_scales<SPW>(p.ws + (int64_t)n * KB, b0 + SPW * rg, KB, sw[i]);
        }
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            if (i < ng) {
                // Stage t has landed once at most min(S - 2, nst - 1 - t)
                // later ones are in flight (loads complete in order).
                wait_stages<S - 2, SPW>(nst - 1 - t);
                asm volatile("" ::: "memory");  // no read of the stage moves above the wait
                if (t + S - 1 < nst) {
                    // slot (t - 1) % S is refilled: its reads must be done
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    issue(t + S - 1);
                }
                const uint8_t *sb = rd + (t % S) * SLOT;
                int4v wf[SPW];
#pragma unroll
                for (int j = 0; j < SPW; ++j)
                    wf[j] = *reinterpret_cast<const int4v *>(sb + (((SPW * rg + j) ^ fsw) << 4));
                auto step = [&](auto jc) {
                    constexpr int J = decltype(jc)::value;
                    if constexpr (J < SPW) {
#pragma unroll
                        for (int f = 0; f < FT; ++f)
                            acc[i][f] = mfma16<XF, (J & 3)>(wf[J], xf[f][J], acc[i][f],
                                                            (int)sw[i][J / 4], (int)sx[f][J / 4]);
                    }
                };
                step(std::integral_constant<int, 0>{});
                step(std::integral_constant<int, 1>{});
                step(std::integral_constant<int, 2>{});
                step(std::integral_constant<int, 3>{});
                step(std::integral_constant<int, 4>{});
                step(std::integral_constant<int, 5>{});
                step(std::integral_constant<int, 6>{});
                step(std::integral_constant<int, 7>{});
                ++t;
            }
        }
    }
    wait_vmcnt<0>();
    __syncthreads();  // every wave is done with its ring: reuse it for the sums

    // 16x16 accumulator layout: lane l, register v holds weight row
    // 4 (l / 16) + v and token l % 16.  red[wave][group][f][token][row].
    float *red = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int i = 0; i < NG; ++i)
        if (i < ng) {
#pragma unroll
            for (int f = 0; f < FT; ++f)
                *reinterpret_cast<f32x4 *>(red + ((wave * NG + i) * FT + f) * 256 + ri * 16 + 4 * rg) =
                    acc[i][f];
        }
    __syncthreads();
    const int cols = ng * 16;
    for (int e = tid; e < cols * M; e += 512) {
        const int nl = e % cols, m = e / cols;
        if (n0 + nl >= N) continue;
        const float *r = red + ((nl >> 4) * FT + (m >> 4)) * 256 + (m & 15) * 16 + (nl & 15);
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) s += r[w * (NG * FT * 256)];
        mx_store_y<YDT>(p.y, (int64_t)m * N + n0 + nl, s);
    }
}

// ---------------------------------------------------------------- launch

template <int XF, int BM, int BN, int WM, int WN, int STA>
static void launch_pp(MxArgs &a, int y_dt, hipStream_t stream) {
    const int tm = (a.M + BM - 1) / BM, tn = (a.N + BN - 1) / BN;
    set_xcd_grid(a, tm, tn, BM, BN);
    const dim3 grid((unsigned)(tm * tn)), block(64 * WM * WN);
    if (y_dt == F32) mx_gemm_pp<XF, BM, BN, WM, WN, STA, F32><<<grid, block, 0, stream>>>(a);
    else if (y_dt == F16) mx_gemm_pp<XF, BM, BN, WM, WN, STA, F16><<<grid, block, 0, stream>>>(a);
    else mx_gemm_pp<XF, BM, BN, WM, WN, STA, BF16><<<grid, block, 0, stream>>>(a);
}

template <int XF>
static void launch_tile(MxArgs &a, int y_dt, hipStream_t stream) {
    const int tm = (a.M + 127) / 128, tn = (a.N + 127) / 128;
    set_xcd_grid(a, tm, tn, 128, 128);
    const dim3 grid((unsigned)(tm * tn));
    if (y_dt == F32) mx_gemm_tile<XF, F32><<<grid, 256, 0, stream>>>(a);
    else if (y_dt == F16) mx_gemm_tile<XF, F16><<<grid, 256, 0, stream>>>(a);
    else mx_gemm_tile<XF, BF16><<<grid, 256, 0, stream>>>(a);
}

template <int XF, int FT, int SPW, int NG, int S>
static void launch_dec_t(MxArgs &a, int y_dt, hipStream_t stream) {
    const dim3 grid((unsigned)((a.N + 16 * a.groups - 1) / (16 * a.groups)));
    if (y_dt == F32) mx_gemm_dec<XF, FT, SPW, NG, S, F32><<<grid, 512, 0, stream>>>(a);
    else if (y_dt == F16) mx_gemm_dec<XF, FT, SPW, NG, S, F16><<<grid, 512, 0, stream>>>(a);
    else mx_gemm_dec<XF, FT, SPW, NG, S, BF16><<<grid, 512, 0, stream>>>(a);
}

template <int XF, int FT>
static void launch_dec(MxArgs &a, int y_dt, hipStream_t stream) {
    // groups of 16 weight rows per block: an equal share for the 256 CUs of
    // as few rounds of blocks as eight groups a block allow
    const int64_t groups = ((int64_t)a.N + 15) / 16;
    const int64_t rounds = (groups + 256 * 8 - 1) / (256 * 8);
    a.groups = (int)((groups + 256 * rounds - 1) / (256 * rounds));
    // the window that lets eight waves cover K, at most 1024 elements (512
    // where the activations of 32 rows would not fit the registers)
    constexpr bool kWide = XF == E2M1 || FT == 1;
    const int spw = a.K <= 1024 ? 1 : a.K <= 2048 ? 2 : a.K <= 4096 || !kWide ? 4 : 8;
    const bool many = a.groups > 2;
    if (spw == 8) {
        if constexpr (kWide) {
            if (many) launch_dec_t<XF, FT, 8, 8, 2>(a, y_dt, stream);
            else launch_dec_t<XF, FT, 8, 2, 2>(a, y_dt, stream);
        }
    } else if (spw == 4) {
        if (many) launch_dec_t<XF, FT, 4, 8, 4>(a, y_dt, stream);
        else launch_dec_t<XF, FT, 4, 2, 3>(a, y_dt, stream);
    } else if (spw == 2) {
        if (many) launch_dec_t<XF, FT, 2, 8, 6>(a, y_dt, stream);
        else launch_dec_t<XF, FT, 2, 2, 3>(a, y_dt, stream);
    } else {
        if (many) launch_dec_t<XF, FT, 1, 8, 8>(a, y_dt, stream);
        else launch_dec_t<XF, FT, 1, 2, 3>(a, y_dt, stream);
    }
}

template <int XF>
static void launch_mx(MxArgs &a, int y_dt, hipStream_t stream, int tile) {
    if (a.M <= 16) return launch_dec<XF, 1>(a, y_dt, stream);
    if (a.M <= 32) return launch_dec<XF, 2>(a, y_dt, stream);
    if (a.K % 128 != 0 || a.K < 256) return launch_tile<XF>(a, y_dt, stream);
    if constexpr (XF == E2M1) {
        if (tile == 0) launch_pp<XF, 256, 256, 4, 2, 2>(a, y_dt, stream);
        else if (tile == 1) launch_pp<XF, 256, 128, 4, 2, 3>(a, y_dt, stream);
        else launch_pp<XF, 128, 128, 2, 2, 2>(a, y_dt, stream);
    } else {
        if (tile == 0) launch_pp<XF, 128, 256, 2, 4, 2>(a, y_dt, stream);
        else launch_pp<XF, 128, 128, 2, 2, 2>(a, y_dt, stream);
    }
}

// The block tile of M > 32: the largest whose tiles fill the 256 CUs best.
static int mx_pick_tile(int x_fmt, int64_t M, int64_t N) {
    struct C { int bm, bn; double eff; int per_cu; };
    const C e2[3] = {{256, 256, 1.0, 1}, {256, 128, 0.85, 1}, {128, 128, 0.7, 2}};
    const C e4[2] = {{128, 256, 1.0, 1}, {128, 128, 0.7, 1}};
    const C *c = x_fmt == E2M1 ? e2 : e4;
    int best = 0;
    double best_score = -1;
    for (int i = 0; i < (x_fmt == E2M1 ? 3 : 2); ++i) {
        const int64_t tiles = ((M + c[i].bm - 1) / c[i].bm) * ((N + c[i].bn - 1) / c[i].bn);
        const int64_t slots = 256 * c[i].per_cu, rounds = (tiles + slots - 1) / slots;
        const double score = (double)tiles / (double)(rounds * slots) * c[i].eff;
        if (score > best_score + 1e-9) { best_score = score; best = i; }
    }
    return best;
}

void launch_gemm_mx(const uint8_t *xq, const uint8_t *xs, int x_fmt, const uint8_t *wq,
                    const uint8_t *ws, int64_t M, int64_t N, int64_t K, void *y, int y_dt,
                    hipStream_t stream, int force_tile) {
    MxArgs a{};
    a.xq = xq; a.xs = xs; a.wq = wq; a.ws = ws;
    a.M = (int)M; a.N = (int)N; a.K = (int)K; a.y = y;
    const int tile = force_tile >= 0 ? force_tile : mx_pick_tile(x_fmt, M, N);
    if (x_fmt == E2M1) launch_mx<E2M1>(a, y_dt, stream, tile);
    else launch_mx<E4M3>(a, y_dt, stream, tile);
}

}  // namespace sq
