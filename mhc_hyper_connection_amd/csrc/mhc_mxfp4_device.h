// mhc_mxfp4_device.h -- microscaled 4-bit floats in registers: 16-bit values to codes and a block
// scale, and back.
//
// A block is 32 consecutive values of a row (the last of a row may be shorter); a value's code
// is e2m1 (0, 1/2, 1, 3/2, 2, 3, 4, 6 and their negatives, sign in bit 3) of its nearest
// multiple of the block's step 2^e, ties to even. With a = the block's largest magnitude, e is the
// least exponent for which a is under 7 steps: a falls on 4 or 6 of them. (From 7 on a would
// be cut to 6; with e one higher it becomes 8 of the smaller steps, its nearest.) So every
// value is off by a fifth of a at most, or by 2^-129 where that is more: e stops at -127, and where
// 6 steps would pass the 16-bit format's range, below that (there off by a quarter of a at
// most). The scale byte is e + 127; 255 marks a block with a NaN or an infinity, whose values
// come back NaN, and whose products are NaN.
// The power of two makes scaling exact, so codes do not depend on how they are computed, and a
// value is exact in the format it came from.
#pragma once

#include "mhc_device.h"

namespace mhc {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
constexpr uint32_t kMxNan = 255;

// Larger of the magnitudes of each 16-bit half (as integers, which order like the values).
__device__ __forceinline__ uint32_t mx_pk_max(uint32_t a, uint32_t b)
{
    typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a),
                                                                  __builtin_bit_cast(u16x2_t, b)));
}
__device__ __forceinline__ uint32_t mx_absmax(u32x4 v)
{
    constexpr uint32_t kAbs = 0x7fff7fffu;
    return mx_pk_max(mx_pk_max(v[0] & kAbs, v[1] & kAbs), mx_pk_max(v[2] & kAbs, v[3] & kAbs));
}
template <int CTRL>
__device__ __forceinline__ uint32_t mx_dpp_max(uint32_t m)
{
    return mx_pk_max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, CTRL, 0xF, 0xF, true));
}
// A block's scale byte from its packed maximum. Adding half of the mantissa's second bit carries
// into the exponent from 1.75 times a power of two on: from 7 steps.
template <bool H>
__device__ __forceinline__ uint32_t mx_scale(uint32_t pk)
{
    const uint32_t lo = pk & 0xffffu, hi = pk >> 16, a = lo > hi ? lo : hi;
    const uint32_t f = __float_as_uint(x16_lo<H>(a));
    const int s = (int)((f + (1u << 21)) >> 23) - 2, most = H ? 140 : 252;
    return a >= (H ? 0x7c00u : 0x7f80u) ? kMxNan : (uint32_t)(s < 0 ? 0 : (s > most ? most : s));
}
// The step as the conversions take it: the power of two's own bits, 2^-127 as the float 2^-127.
__device__ __forceinline__ float mx_step(uint32_t scale)
{
    return __uint_as_float(scale == 0 ? 1u << 22 : scale << 23);
}
// Eight 16-bit values to a word of codes, the first in the low bits.
template <bool H>
__device__ __forceinline__ uint32_t mx_encode(u32x4 v, uint32_t scale)
{
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
    const float step = mx_step(scale == kMxNan ? 127u : scale);
    const uint32_t w[4] = {v[0], v[1], v[2], v[3]};   // a vector's element is not taken for a value of its own by a bit cast
    uint32_t c = 0;
    if constexpr (H) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, w[0]), step, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, w[1]), step, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, w[2]), step, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, w[3]), step, 3);
    } else {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[0]), step, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[1]), step, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[2]), step, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[3]), step, 3);
    }
    return scale == kMxNan ? 0u : c;
}
// A word of codes to eight 16-bit values. Through fp32, whose product with the step is exact (a
// subnormal one too), and which the 16-bit format then holds exactly where the codes came from it.
template <bool H>
__device__ __forceinline__ u32x4 mx_decode(uint32_t c, uint32_t scale)
{
    const float step = scale == kMxNan ? __builtin_nanf("") : mx_step(scale);
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        typedef float f32x2_t __attribute__((ext_vector_type(2)));
        f32x2_t f;
        if (e == 0) f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 0);
        else if (e == 1) f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 1);
        else if (e == 2) f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 2);
        else f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 3);
        const float lo = f[0] * step, hi = f[1] * step;
        v[e] = pack_x16<H>(lo, hi);
    }
    return v;
}

}  // namespace
}  // namespace mhc
