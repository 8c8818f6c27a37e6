// Device-side helpers of the microscaled (MX) cache of keys and values
// (include/sq_kv.h): where a token's rows lie, and codes as values of the type
// that the consumer computes in.
#pragma once

#include "mx_device.h"
#include "sq_kv_launch.h"

namespace sq {

// The row (of codes or of scales) of a head's token at place `at` of a page.
__device__ __forceinline__ int64_t kv_row(const KvCache &c, int64_t page, int head, int at) {
    return ((page * c.heads + head) << c.page_log) + at;
}

// Sequence of a dense row: the last b with cu[b] <= row (empty sequences lie
// before it).  cu[0] <= row < cu[B].
__device__ __forceinline__ int kv_find(const int32_t *cu, int B, int64_t row) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= row) lo = mid;
        else hi = mid;
    }
    return lo;
}

// An E8M0 byte as the scale operand of the conversions below: they take the
// operand's exponent, so 0 gives 2^-127 and 255 gives NaN, as the format says.
__device__ __forceinline__ float e8m0(uint32_t e) { return __uint_as_float(e << 23); }

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Two e2m1 codes of byte B of a word, or two e4m3 codes of half H, as values
// of a 16-bit type (one word), rounded to nearest even.
template <int DT, int B>
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t w, float s) {
    if constexpr (DT == BF16)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, B));
    else
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, B));
}
template <int DT, bool H>
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w, float s) {
    if constexpr (DT == BF16)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, H));
    else
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, s, H));
}

// Eight successive elements' codes (one word of e2m1, two of e4m3) as four
// words of a 16-bit type.
template <int FMT, int DT>
__device__ __forceinline__ uint4 codes8_to_16(const uint32_t *w, float s) {
    uint4 r;
    if constexpr (FMT == E2M1) {
        r.x = e2m1_pair<DT, 0>(w[0], s);
        r.y = e2m1_pair<DT, 1>(w[0], s);
        r.z = e2m1_pair<DT, 2>(w[0], s);
        r.w = e2m1_pair<DT, 3>(w[0], s);
    } else {
        r.x = e4m3_pair<DT, false>(w[0], s);
        r.y = e4m3_pair<DT, true>(w[0], s);
        r.z = e4m3_pair<DT, false>(w[1], s);
        r.w = e4m3_pair<DT, true>(w[1], s);
    }
    return r;
}

}  // namespace sq
