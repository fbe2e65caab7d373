// mx_items.h -- blocks of a cache held in 8 or 4 bits (gfx950).
//
// 32 values along a head share a byte e, which stands for 2^(e - 127) (255: NaN); a value is a code, e4m3 or e2m1, times that.
// The conversions below are the CDNA4 instructions for exactly these formats: powers of two change no digit, so what
// they give is exact wherever the type has the number, else rounded once (next to its smallest number, and infinite past its largest one).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "drafted_plan.h"

namespace moe {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short mx_s16x2 __attribute__((ext_vector_type(2)));

// 16 loaded bytes as the 16-bit values that they stand for, whose block's scale byte is e. MX_NONE: as they are.
template <bool F16, int FMT> __device__ __forceinline__ void mx_expand(const u32x4 &r, uint32_t e, u32x4 *x) {
    if constexpr (FMT == MX_NONE) {
        x[0] = r;
    } else {
        const float s = __uint_as_float(e << 23);
#define MX_PAIR8(W, HI)                                                                                       \
    (F16 ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(W, s, HI))                   \
         : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(W, s, HI)))
#define MX_PAIR4(W, BYTE)                                                                                     \
    (F16 ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(W, s, BYTE))                 \
         : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(W, s, BYTE)))
        if constexpr (FMT == MX_E4M3) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                x[i] = u32x4{MX_PAIR8(r[2 * i], false), MX_PAIR8(r[2 * i], true), MX_PAIR8(r[2 * i + 1], false),
                             MX_PAIR8(r[2 * i + 1], true)};
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = u32x4{MX_PAIR4(r[i], 0), MX_PAIR4(r[i], 1), MX_PAIR4(r[i], 2), MX_PAIR4(r[i], 3)};
        }
#undef MX_PAIR8
#undef MX_PAIR4
    }
}

// The scale byte of a block whose largest magnitude is `top`: of the smallest power of two, 2^-126 at least, under which it
// does not pass the largest code (448 or 6); 255 where it is not finite. The power stops where the largest code is still
// finite in the rows' type (2^119 and 2^125 in bf16, 2^7 and 2^13 in f16), and what is larger takes the largest code.
template <bool F16, int FMT> constexpr uint32_t mx_last_scale() { return (F16 ? 142 : 254) - (FMT == MX_E4M3 ? 8 : 2); }
template <bool F16, int FMT> __device__ __forceinline__ uint32_t mx_scale(float top) {
    constexpr int EMAX = FMT == MX_E4M3 ? 8 : 2;                              // exponent of the largest code
    constexpr uint32_t FRACTION = FMT == MX_E4M3 ? 0x600000u : 0x400000u;     // and its fraction, 1.75 and 1.5
    const uint32_t bits = __float_as_uint(top) & 0x7FFFFFFFu;
    if (bits >= 0x7F800000u) return 255;
    const int e = (int)(bits >> 23) - EMAX + ((bits & 0x7FFFFFu) > FRACTION ? 1 : 0);
    return (uint32_t)min(max(e, 1), (int)mx_last_scale<F16, FMT>());
}

// Eight values of a block with scale byte e as codes, to nearest even: 8 bytes, or 4 in the first word.
template <int FMT> __device__ __forceinline__ uint2 mx_codes(const float *x, uint32_t e) {
    if (e == 255) return make_uint2(0, 0);       // the scale alone makes the block NaN
    const float s = __uint_as_float(e << 23);
    if constexpr (FMT == MX_E4M3) {
        uint2 r;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mx_s16x2 w = {0, 0};
            w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, x[4 * i], x[4 * i + 1], s, false);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, x[4 * i + 2], x[4 * i + 3], s, true);
            (i ? r.y : r.x) = __builtin_bit_cast(uint32_t, w);
        }
        return r;
    } else {
        uint32_t w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], s, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], s, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], s, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], s, 3);
        return make_uint2(w, 0);
    }
}

}  // namespace moe
