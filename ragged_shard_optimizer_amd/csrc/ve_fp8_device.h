// ve_fp8_device.h -- the 8-bit floating-point code: a block's scale exponent,
// codes of fp32 values, and back.
#pragma once

#include "ve_linear_device.h"

namespace ve {

// Largest magnitude of the finite values, kept as the bits of |v|; `bad`
// collects whether any was infinite or NaN.
__device__ __forceinline__ uint32_t finite_amax(uint32_t m, float v, bool& bad) {
    const uint32_t a = __float_as_uint(v) & 0x7fffffffu;
    const bool f = a < 0x7f800000u;
    bad |= !f;
    return f && a > m ? a : m;
}

// The smallest e >= -127 with amax <= MAX 2^e, plus 127, from the bits of
// amax.  MAX is 1.75 2^8 (E4M3) or 1.75 2^15 (E5M2): the exponent of amax, one
// more where its mantissa is above 1.75, less 8 or 15.
__device__ __forceinline__ uint32_t fp8_exponent(uint32_t amax, int format) {
    const int e = (int)((amax + 0x1fffffu) >> 23) - (format == VE_E4M3 ? 8 : 15);
    return (uint32_t)max(e, 0);
}
// 2^-e of a stored exponent (at most 247, so that this is a normal number).
__device__ __forceinline__ float fp8_inverse(uint32_t e) { return __uint_as_float((254u - e) << 23); }
// 2^e (e = 255: NaN).
__device__ __forceinline__ float fp8_scale(uint32_t e) {
    return e == 0 ? 0x1p-127f : __uint_as_float(e == 255 ? 0x7fc00000u : e << 23);
}

// Codes of 8 values of one block: the product with a power of two is exact but
// where it falls below fp32's range, far below the formats' smallest value,
// and the conversion rounds to nearest even.  No finite value passes MAX.
// Infinities and NaN (bad: there may be some) are written by hand, so that
// they do not depend on the conversion's mode.
__device__ __forceinline__ u32x2 fp8_encode8(const float* v, float inv, int format, bool bad) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float s[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) s[t] = v[4 * h + t] * inv;
        int p = 0;
        if (format == VE_E4M3) {
            p = __builtin_amdgcn_cvt_pk_fp8_f32(s[0], s[1], p, false);
            p = __builtin_amdgcn_cvt_pk_fp8_f32(s[2], s[3], p, true);
        } else {
            p = __builtin_amdgcn_cvt_pk_bf8_f32(s[0], s[1], p, false);
            p = __builtin_amdgcn_cvt_pk_bf8_f32(s[2], s[3], p, true);
        }
        w[h] = (uint32_t)p;
    }
    if (bad) {
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const uint32_t b = __float_as_uint(v[t]), a = b & 0x7fffffffu;
            if (a < 0x7f800000u) continue;
            const uint32_t c = (b >> 24 & 0x80u) | (format == VE_E5M2 && a == 0x7f800000u ? 0x7cu : 0x7fu);
            w[t >> 2] = (w[t >> 2] & ~(255u << (8 * (t & 3)))) | c << (8 * (t & 3));
        }
    }
    return u32x2{w[0], w[1]};
}

// The values of 4 codes.
__device__ __forceinline__ void fp8_decode4(uint32_t w, int format, float* v) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    f32x2 lo, hi;
    if (format == VE_E4M3) {
        lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
        hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    } else {
        lo = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, false);
        hi = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, true);
    }
    v[0] = lo[0]; v[1] = lo[1]; v[2] = hi[0]; v[3] = hi[1];
}

}  // namespace ve
