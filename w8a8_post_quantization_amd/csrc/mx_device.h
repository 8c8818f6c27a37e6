// Device-side helpers of the microscaled (MX) kernels: eight elements a lane,
// four neighbouring lanes (a quad) a block of 32, one E8M0 scale a block.
// (include/sq_mx.h has the formats and the quantizer's definition.)
#pragma once

#include "sq_device.h"

namespace sq {

enum MxFmt { E2M1 = 0, E4M3 = 1 };

typedef short short2v __attribute__((ext_vector_type(2)));

// Eight successive elements as loaded: 16 bytes (16-bit types) or 32 (fp32).
template <int DT> struct Raw8 { uint4 v[DT == F32 ? 2 : 1]; };

template <int DT, bool NTL>
__device__ __forceinline__ Raw8<DT> load8(const void *x, int64_t i8) {
    constexpr int W = DT == F32 ? 2 : 1;
    const uint4 *p = reinterpret_cast<const uint4 *>(x) + i8 * W;
    Raw8<DT> r;
#pragma unroll
    for (int i = 0; i < W; ++i) r.v[i] = ld16<NTL>(p + i);
    return r;
}

// The halves of a word of two fp16 as fp32, exactly: h * 1 + -0 (-0 stays -0).
// The plain conversion issues slower (layer norm of 16384 x 7168: 71 us with it,
// 68 so).
__device__ __forceinline__ void widen_f16(uint32_t w, float &lo, float &hi) {
    asm("v_fma_mix_f32 %0, %1, 1.0, neg(0) op_sel_hi:[1,0,0]" : "=v"(lo) : "v"(w));
    asm("v_fma_mix_f32 %0, %1, 1.0, neg(0) op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(hi) : "v"(w));
}

template <int DT>
__device__ __forceinline__ void widen8(const Raw8<DT> &r, float (&out)[8]) {
    if constexpr (DT == F16) {
        widen_f16(r.v[0].x, out[0], out[1]);
        widen_f16(r.v[0].y, out[2], out[3]);
        widen_f16(r.v[0].z, out[4], out[5]);
        widen_f16(r.v[0].w, out[6], out[7]);
        return;
    }
    widen16<DT>(r.v[0], out);
    if constexpr (DT == F32) widen16<DT>(r.v[1], out + 4);
}

__device__ __forceinline__ void load_f32x8(const float *p, float (&m)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0];
    const float4 b = reinterpret_cast<const float4 *>(p)[1];
    m[0] = a.x; m[1] = a.y; m[2] = a.z; m[3] = a.w;
    m[4] = b.x; m[5] = b.y; m[6] = b.z; m[7] = b.w;
}

// The larger magnitude of the lane and its quad neighbours, as the bits of
// |v|: unsigned bits order magnitudes, and an infinity or NaN stays on top
// (a float max would drop the NaN).
__device__ __forceinline__ uint32_t quad_max(uint32_t b) {
    const uint32_t o1 = (uint32_t)__builtin_amdgcn_mov_dpp((int)b, 0xb1, 0xf, 0xf, true);
    b = b > o1 ? b : o1;
    const uint32_t o2 = (uint32_t)__builtin_amdgcn_mov_dpp((int)b, 0x4e, 0xf, 0xf, true);
    return b > o2 ? b : o2;
}

// Eight fp32 values of a lane -> their codes (4 bytes of e2m1, 8 of e4m3) and
// the block's scale byte (the same in the four lanes of the quad).  All 64
// lanes of the wave call it.
template <int FMT> struct MxCodes { uint32_t w[FMT == E2M1 ? 1 : 2]; };

template <int FMT>
__device__ __forceinline__ MxCodes<FMT> mx_encode8(const float (&v)[8], uint32_t &e_out) {
    // the largest |v| of the lane, a NaN if there is one (IEEE maximum: three
    // operands and their magnitudes an instruction)
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = __builtin_elementwise_maximum(top, __builtin_fabsf(v[i]));
    const uint32_t b = quad_max(__float_as_uint(top) & 0x7fffffffu);
    constexpr int P = FMT == E2M1 ? 2 : 8;
    const int E = (int)(b >> 23);
    const int e = E > P ? E - P : 0;
    const bool finite = E != 255;
    e_out = finite ? (uint32_t)e : 255u;
    // 2^(e - 127) as fp32 (e = 0: the subnormal 2^-127)
    const float s = __uint_as_float(e > 0 ? (uint32_t)e << 23 : 0x00400000u);
    MxCodes<FMT> c;
    if constexpr (FMT == E2M1) {
        // round to nearest even of v / s, saturating (the instruction)
        int w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], s, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
        c.w[0] = finite ? (uint32_t)w : 0u;
    } else {
        // the e4m3 conversion turns magnitudes above 464 into NaN: clamp to
        // 448 s = 1.75 2^(e - 119) first
        const float lim = __uint_as_float(((uint32_t)(e + 8) << 23) | 0x00600000u);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] = __builtin_amdgcn_fmed3f(v[4 * h + i], -lim, lim);
            short2v w = {0, 0};
            w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, z[0], z[1], s, false);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, z[2], z[3], s, true);
            c.w[h] = finite ? __builtin_bit_cast(uint32_t, w) : 0u;
        }
    }
    return c;
}

// Store the codes of the i8-th group of eight elements, and by the quad's
// first lane the scale byte of its block.
template <int FMT, bool NTS>
__device__ __forceinline__ void mx_store8(uint8_t *q, uint8_t *scale, int64_t i8,
                                          const MxCodes<FMT> &c, uint32_t e) {
    if constexpr (FMT == E2M1) {
        uint32_t *p = reinterpret_cast<uint32_t *>(q) + i8;
        if constexpr (NTS) __builtin_nontemporal_store(c.w[0], p);
        else *p = c.w[0];
    } else {
        typedef unsigned int u2v __attribute__((ext_vector_type(2)));
        u2v *p = reinterpret_cast<u2v *>(q) + i8;
        const u2v v = {c.w[0], c.w[1]};
        if constexpr (NTS) __builtin_nontemporal_store(v, p);
        else *p = v;
    }
    if ((threadIdx.x & 3) == 0) scale[i8 >> 2] = (uint8_t)e;
}

}  // namespace sq
