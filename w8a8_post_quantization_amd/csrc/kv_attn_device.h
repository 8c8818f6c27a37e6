// What the attention kernels over the microscaled cache share: a sequence's
// keys and queries, the matrix instructions by type, non-finite values.
#pragma once

#include "kv_device.h"
#include "pipe_device.h"

namespace sq {

// For a kernel's lambdas: left as calls, they would have its registers in memory.
#define SQ_INLINE __attribute__((always_inline))

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Finite, and below every score: the running maximum of a row that has seen no
// key yet.
constexpr float kNoMax = -3.402823466e38f;

// Weights are 2^(score - m), rounded to the queries' type, in which the matrix
// instructions take both operands (their sum is of the unrounded ones, in fp32;
// the output's error is 2.2e-3 of its norm in bf16 and 2.9e-4 in fp16, of which
// its own rounding is 1.7e-3 and 2.1e-4).  m is set to a row's largest score less kLift, and
// may trail the true one by kTrail more before the row is rescaled: rescaling is
// rare.  fp16 holds 2^-14 .. 2^15 in full and nothing below 2^-25, so its weights
// are lifted to the upper end, 2^(kTrail + kLift) = 2^15 at the most: those of
// 2^-21 of the largest have all their bits, those of 2^-32 are lost (unlifted,
// 3500 keys of 2^-26 each, 18 nats below the first, came out up to 10 bounds
// off).  bf16 has fp32's range.  (The difference of score and m is compared, not m
// plus the slack: where fp32's step is 16 that sum is rounded to the next score,
// whose weight would be 2^16.)
constexpr float kTrail = 8.0f;
template <int DT> constexpr float kLift = DT == F16 ? 7.0f : 0.0f;

// C += A B of 16 x 16 x 32: lane l holds A[l % 16][8 (l / 16) ..], B[..][l % 16]
// of the same eight inner indices, C[4 (l / 16) ..][l % 16].
template <int DT>
__device__ __forceinline__ f32x4 mfma16(const uint4 &a, const uint4 &b, f32x4 c) {
    if constexpr (DT == BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// The same of 32 x 32 x 16: A[l % 32][8 (l / 32) ..], B[..][l % 32], C[i % 4 +
// 8 (i / 4) + 4 (l / 32)][l % 32].
template <int DT>
__device__ __forceinline__ f32x16 mfma32(const uint4 &a, const uint4 &b, f32x16 c) {
    if constexpr (DT == BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// A direct-to-LDS load of 4 bytes a lane (pipe_device.h), to lds_base + 4 lane.
__device__ __forceinline__ void lds_dma4(const void *g, uint32_t lds_base) {
    asm volatile(
        "s_mov_b32 m0, %1\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dword %0, off"
        :
        : "v"(g), "s"(lds_base)
        : "memory", "m0");
}

// Two fp32 -> one word of the 16-bit type, to nearest even.
template <int DT>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if constexpr (DT == BF16) {
        const bf16x2 v = {(__bf16)lo, (__bf16)hi};
        return __builtin_bit_cast(uint32_t, v);
    } else {
        const f16x2 v = {(_Float16)lo, (_Float16)hi};
        return __builtin_bit_cast(uint32_t, v);
    }
}

// One half of a word of two 16-bit values, as fp32.
template <int DT>
__device__ __forceinline__ float half_of(uint32_t w, int h) {
    if constexpr (DT == BF16) return __uint_as_float(h ? w & 0xffff0000u : w << 16);
    else return (float)__builtin_bit_cast(f16x2, w)[h];
}

// Words that hold N bytes of codes, as loaded.
template <int N> struct Words { uint32_t w[N < 4 ? 1 : N / 4]; };
template <int N>
__device__ __forceinline__ Words<N> load_codes(const uint8_t *p) {
    Words<N> r;
    if constexpr (N == 2) {
        r.w[0] = *reinterpret_cast<const uint16_t *>(p);
    } else if constexpr (N == 4) {
        r.w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (N == 8) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        r.w[0] = v.x;
        r.w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N / 16; ++i) {
            const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
            r.w[4 * i] = v.x;
            r.w[4 * i + 1] = v.y;
            r.w[4 * i + 2] = v.z;
            r.w[4 * i + 3] = v.w;
        }
    }
    return r;
}

// The q-th pair of codes among a lane's words.
template <int FMT, int DT, int N>
__device__ __forceinline__ uint32_t pair_of(const Words<N> &c, int q, float s) {
    if constexpr (FMT == E2M1) {
        const uint32_t w = c.w[q >> 2];
        switch (q & 3) {
            case 0: return e2m1_pair<DT, 0>(w, s);
            case 1: return e2m1_pair<DT, 1>(w, s);
            case 2: return e2m1_pair<DT, 2>(w, s);
            default: return e2m1_pair<DT, 3>(w, s);
        }
    } else {
        return q & 1 ? e4m3_pair<DT, true>(c.w[q >> 1], s) : e4m3_pair<DT, false>(c.w[q >> 1], s);
    }
}

// Whether a value of a block with this scale byte may be infinite or NaN in the
// type (6 2^(e - 127) or 448 2^(e - 127) past its largest), or one of the codes
// is a NaN (e4m3; the quantizer makes none).
template <int FMT, int DT, int N>
__device__ __forceinline__ bool may_be_nonfinite(const Words<N> &c, uint32_t e) {
    constexpr uint32_t kFrom = DT == BF16 ? (FMT == E2M1 ? 253 : 247) : (FMT == E2M1 ? 141 : 135);
    bool any = e >= kFrom;
    if constexpr (FMT == E4M3) {
#pragma unroll
        for (int i = 0; i < (N + 3) / 4; ++i) any |= (((c.w[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
    }
    return any;
}

// One sequence's part in the call.  lo .. hi: the keys that any query sees.
struct KvSeq {
    int q0, nq, nk, lo, hi;
    bool over;  // longer than its row of the table: its queries get NaN
};

__device__ __forceinline__ KvSeq kv_seq(const KvAttention &a, int b) {
    KvSeq s;
    const int T = (int)a.T;
    int q0 = b, q1 = b + 1;
    if (a.cu_q) {
        q0 = a.cu_q[b];
        q1 = a.cu_q[b + 1];
        q0 = q0 < 0 ? 0 : q0 > T ? T : q0;
        q1 = q1 < q0 ? q0 : q1 > T ? T : q1;
    }
    s.q0 = q0;
    s.nq = q1 - q0;
    const int cap = (int)(a.width << a.cache.page_log);
    const int len = a.seq_lens[b];
    s.over = len > cap;
    s.nk = len < 0 ? 0 : s.over ? cap : len;
    s.hi = s.nk;
    const int64_t lo = a.window ? (int64_t)s.nk - s.nq + 1 - a.window : 0;
    s.lo = lo > 0 ? (int)lo : 0;
    return s;
}

// The keys that a sequence's query i sees end here (none: 0 or less).
__device__ __forceinline__ int keys_end(const KvAttention &a, const KvSeq &s, int i) {
    return a.causal ? s.nk - s.nq + i + 1 : s.nk;
}

// What a row's weighted values are multiplied by, `end` its keys_end.  No key
// seen gives 0; of a row that sees some, the weights sum to 0 only where every
// score is -inf: 0 / 0.
__device__ __forceinline__ float row_factor(float sum, int end, bool over) {
    if (over || (end > 0 && sum == 0.0f)) return __uint_as_float(0x7fc00000u);
    return end > 0 ? 1.0f / sum : 0.0f;
}

}  // namespace sq
