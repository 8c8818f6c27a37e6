// Building blocks of the pipelined matrix kernels: the tile-to-block mapping,
// direct-to-LDS loads, the waits and barrier of an LDS ring, and the
// instruction pattern of a stage.
#pragma once

#include "sq_device.h"

namespace sq {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int int8x __attribute__((ext_vector_type(8)));

__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// The tiles of a product's outputs and their deal to the XCDs.
struct TileGrid {
    int tiles_n;
    int tiles_m;
    int xcd_gm, xcd_gn;  // XCD grid of the tile mapping (tile_of), or 0: row-major
};

// The tile of block b.  The hardware deals a kernel's blocks to the 8 XCDs
// round-robin (block b to XCD b % 8), and each XCD has its own L2.  With an
// XCD grid gm x gn (gm | tiles_m, gn | tiles_n, gm gn = 8) XCD x takes the
// tiles of one sub-rectangle (tiles_m / gm) x (tiles_n / gn) of the tile
// grid, row-major, so it fetches only those activation rows and weight rows
// instead of most of both.  Any mapping gives the same results (a
// bijection of tiles); only the cache traffic changes.
__device__ __forceinline__ void tile_of(const TileGrid &p, int b, int &tm, int &tn) {
    if (p.xcd_gm == 0) {
        tm = b / p.tiles_n;
        tn = b % p.tiles_n;
        return;
    }
    const int x = b & 7, j = b >> 3;
    const int rm = p.tiles_m / p.xcd_gm, rn = p.tiles_n / p.xcd_gn;
    tm = (x / p.xcd_gn) * rm + j / rn;
    tn = (x % p.xcd_gn) * rn + j % rn;
}

// XCD grid for tile_of: the factorization gm x gn = 8 (gm | tm, gn | tn)
// that fetches the fewest operand bytes per XCD, rm BM + rn BN rows of K
// bytes; none (row-major order) when the tiles do not split 8 ways.
inline void set_xcd_grid(TileGrid &a, int tm, int tn, int bm, int bn) {
    a.tiles_m = tm;
    a.tiles_n = tn;
    a.xcd_gm = a.xcd_gn = 0;
    long best = -1;
    for (int gm = 1; gm <= 8; gm *= 2) {
        const int gn = 8 / gm;
        if (tm % gm || tn % gn) continue;
        const long cost = (long)(tm / gm) * bm + (long)(tn / gn) * bn;
        if (best < 0 || cost < best) {
            best = cost;
            a.xcd_gm = gm;
            a.xcd_gn = gn;
        }
    }
}

typedef __attribute__((address_space(3))) void lds_void_t;

// One direct-to-LDS load: 16 bytes per lane from `g` into LDS at
// lds_base + 16 * lane (lds_base wave-uniform, in M0).  Written as inline
// asm on purpose: the compiler treats every later LDS read as possibly
// aliasing an LDS write that is still in flight from the builtin form and
// waits for all of them (vmcnt(0)) before the read, which drains the whole
// prefetch ring each stage.  Here the kernel's own vmcnt waits and
// barriers order the ring.  The instruction has no register results; its
// address operands are read when it issues.  s_nop covers the M0-write ->
// LDS-DMA hazard.
__device__ __forceinline__ void lds_dma16(const void *g, uint32_t lds_base) {
    asm volatile(
        "s_mov_b32 m0, %1\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %0, off"
        :
        : "v"(g), "s"(lds_base)
        : "memory", "m0");
}

// The same with the nontemporal hint, for data read once (a weight stream
// that should not displace reused lines in the caches).
__device__ __forceinline__ void lds_dma16_nt(const void *g, uint32_t lds_base) {
    asm volatile(
        "s_mov_b32 m0, %1\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %0, off nt"
        :
        : "v"(g), "s"(lds_base)
        : "memory", "m0");
}

// NL (1..4) direct-to-LDS loads under one M0 write: load j moves 16 bytes
// per lane from g[j] into LDS at lds_base + 1024 j + 16 lane.  The
// instruction offset (1024 j) is added to both the global and the LDS
// address, so g[j] is passed biased by -1024 j.  Rewriting M0 before every
// load makes each wave wait for its previous load to be accepted: measured
// on this GPU from an L2-resident source, 4 waves per CU moved 23 B/clk with
// one M0 write per load and 51.5 B/clk (the vector L1's rate for coalesced
// register loads) with one per four loads.  (The GEMMs here issue few
// enough loads per stage that their times did not change.)  NT adds the
// nontemporal hint.
template <int NL, bool NT>
__device__ __forceinline__ void lds_dma_group(const int8_t *const *g, uint32_t lds_base) {
    static_assert(NL >= 1 && NL <= 4, "one M0 covers 4 KB of instruction offsets");
    const int8_t *b0 = g[0];
    const int8_t *b1 = NL > 1 ? g[1] - 1 * 1024 : nullptr;
    const int8_t *b2 = NL > 2 ? g[2] - 2 * 1024 : nullptr;
    const int8_t *b3 = NL > 3 ? g[3] - 3 * 1024 : nullptr;
#define SQ_DMA_ASM(HINT)                                                                   \
    if constexpr (NL == 1) {                                                               \
        asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\t"                                    \
                     "global_load_lds_dwordx4 %0, off" HINT                                \
                     : : "v"(b0), "s"(lds_base) : "memory", "m0");                         \
    } else if constexpr (NL == 2) {                                                        \
        asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\t"                                    \
                     "global_load_lds_dwordx4 %0, off" HINT "\n\t"                        \
                     "global_load_lds_dwordx4 %1, off offset:0x400" HINT                    \
                     : : "v"(b0), "v"(b1), "s"(lds_base) : "memory", "m0");                \
    } else if constexpr (NL == 3) {                                                        \
        asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\t"                                    \
                     "global_load_lds_dwordx4 %0, off" HINT "\n\t"                        \
                     "global_load_lds_dwordx4 %1, off offset:0x400" HINT "\n\t"            \
                     "global_load_lds_dwordx4 %2, off offset:0x800" HINT                    \
                     : : "v"(b0), "v"(b1), "v"(b2), "s"(lds_base) : "memory", "m0");       \
    } else {                                                                               \
        asm volatile("s_mov_b32 m0, %4\n\ts_nop 0\n\t"                                    \
                     "global_load_lds_dwordx4 %0, off" HINT "\n\t"                        \
                     "global_load_lds_dwordx4 %1, off offset:0x400" HINT "\n\t"            \
                     "global_load_lds_dwordx4 %2, off offset:0x800" HINT "\n\t"            \
                     "global_load_lds_dwordx4 %3, off offset:0xc00" HINT                    \
                     : : "v"(b0), "v"(b1), "v"(b2), "v"(b3), "s"(lds_base)                  \
                     : "memory", "m0");                                                    \
    }
    if constexpr (NT) {
        SQ_DMA_ASM(" nt")
    } else {
        SQ_DMA_ASM("")
    }
#undef SQ_DMA_ASM
}

// Loads j = 0 .. N-1 of a stage into consecutive 1 KB LDS blocks, M0 set
// once per four.
template <int N, bool NT>
__device__ __forceinline__ void lds_dma_run(const int8_t *const *g, uint32_t lds_base) {
#pragma unroll
    for (int j0 = 0; j0 < N; j0 += 4) {
        if (N - j0 >= 4) lds_dma_group<4, NT>(g + j0, lds_base + (uint32_t)(j0 * 1024));
        else if (N - j0 == 3) lds_dma_group<3, NT>(g + j0, lds_base + (uint32_t)(j0 * 1024));
        else if (N - j0 == 2) lds_dma_group<2, NT>(g + j0, lds_base + (uint32_t)(j0 * 1024));
        else lds_dma_group<1, NT>(g + j0, lds_base + (uint32_t)(j0 * 1024));
    }
}

// The same from a wave-uniform base and a 32-bit offset per lane (one register
// a load instead of two, and the stage's advance is scalar): load j moves 16
// bytes (B = 4: 4 bytes) per lane from base + off[j] into LDS at lds_base +
// 64 B j + B lane.  off[j] holds the true offset plus dma_bias<B>(j), which the
// base is lowered by kDmaBias for: the instruction's own offset (64 B j, for
// LDS) is added to the address too, and a lane's offset cannot be negative.
constexpr uint32_t kDmaBias = 4096;
template <int B>
__device__ __forceinline__ uint32_t dma_bias(int j) {
    return kDmaBias - (uint32_t)(64 * B * (j & 3));
}
template <int N, int B, bool NT>
__device__ __forceinline__ void lds_dma_based(const uint32_t *off, const void *base,
                                              uint32_t lds_base) {
    static_assert(B == 16 || B == 4, "bytes per lane");
    const uint64_t sb = (uint64_t)base - kDmaBias;
#define SQ_DMA_BASED(OP, HINT, O1, O2, O3)                                                       \
    if (N - j0 >= 4) {                                                                           \
        asm volatile("s_mov_b32 m0, %5\n\ts_nop 0\n\t" OP " %0, %4" HINT "\n\t" OP               \
                     " %1, %4 offset:" O1 HINT "\n\t" OP " %2, %4 offset:" O2 HINT "\n\t" OP     \
                     " %3, %4 offset:" O3 HINT                                                   \
                     : : "v"(off[j0]), "v"(off[j0 + 1]), "v"(off[j0 + 2]), "v"(off[j0 + 3]),     \
                       "s"(sb), "s"(lds_base + (uint32_t)(64 * B * j0)) : "memory", "m0");       \
    } else if (N - j0 == 3) {                                                                    \
        asm volatile("s_mov_b32 m0, %4\n\ts_nop 0\n\t" OP " %0, %3" HINT "\n\t" OP               \
                     " %1, %3 offset:" O1 HINT "\n\t" OP " %2, %3 offset:" O2 HINT               \
                     : : "v"(off[j0]), "v"(off[j0 + 1]), "v"(off[j0 + 2]), "s"(sb),              \
                       "s"(lds_base + (uint32_t)(64 * B * j0)) : "memory", "m0");                \
    } else if (N - j0 == 2) {                                                                    \
        asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\t" OP " %0, %2" HINT "\n\t" OP               \
                     " %1, %2 offset:" O1 HINT                                                   \
                     : : "v"(off[j0]), "v"(off[j0 + 1]), "s"(sb),                                \
                       "s"(lds_base + (uint32_t)(64 * B * j0)) : "memory", "m0");                \
    } else {                                                                                     \
        asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\t" OP " %0, %1" HINT                         \
                     : : "v"(off[j0]), "s"(sb), "s"(lds_base + (uint32_t)(64 * B * j0))          \
                     : "memory", "m0");                                                          \
    }
#pragma unroll
    for (int j0 = 0; j0 < N; j0 += 4) {
        if constexpr (B == 4) {
            static_assert(!NT, "no nontemporal form");
            SQ_DMA_BASED("global_load_lds_dword", "", "0x100", "0x200", "0x300")
        } else if constexpr (NT) {
            SQ_DMA_BASED("global_load_lds_dwordx4", " nt", "0x400", "0x800", "0xc00")
        } else {
            SQ_DMA_BASED("global_load_lds_dwordx4", "", "0x400", "0x800", "0xc00")
        }
    }
#undef SQ_DMA_BASED
}

// s_waitcnt vmcnt(N) leaving lgkmcnt / expcnt alone (gfx9 encoding).
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// Wait until at most `later` stages of P loads each are in flight
// (later <= L, or negative for none; vmcnt takes an immediate, hence the
// unrolled choice).
template <int L, int P>
__device__ __forceinline__ void wait_stages(int later) {
    if constexpr (L == 0) {
        wait_vmcnt<0>();
    } else {
        if (later >= L) wait_vmcnt<L * P>();
        else wait_stages<L - 1, P>(later);
    }
}

// Workgroup barrier for the LDS ring only.  __syncthreads() carries a
// release fence that waits for every outstanding global load (vmcnt(0)),
// which would drain the in-flight stages; here each wave has already waited
// for its own stage loads with vmcnt(N), and only LDS traffic must be
// complete before the barrier.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Scheduling pattern after the stage barrier: each MFMA is followed by one
// DS read (while any remain) and its share of the stage's direct loads.
template <int MQ, int RQ, int L, int R>
__device__ __forceinline__ void sched_tail() {
    if constexpr (R < MQ) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 1);  // MFMA
        if constexpr (R < RQ) __builtin_amdgcn_sched_group_barrier(0x100, 1, 1);  // DS read
        constexpr int per = (L + MQ - 1) / MQ;
        constexpr int left = L - R * per;
        if constexpr (left > 0)
            __builtin_amdgcn_sched_group_barrier(0x020, left < per ? left : per, 1);  // VMEM read
        sched_tail<MQ, RQ, L, R + 1>();
    }
}

}  // namespace sq
