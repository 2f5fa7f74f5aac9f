// mhc_ckpt_device.h -- the 8-bit checkpoint format in registers: 16-bit values to codes and
// a block scale, and back.
//
// A block is 32 consecutive values of a row (the last of a row may be shorter). With
// a = the largest magnitude in it, its step is 2^e, e = floor(log2 a) - 6 (at least -24 for
// fp16, whose least value is 2^-24, and -126 for bf16, the least exponent of a normal
// float), and a value's code is its nearest multiple of the step, ties to even, within
// +-127. So a falls on 64 .. 127 steps (on fewer at the least step), every value is off by
// half a step at most (those above 127.5 steps by less than one): by a/128, or by 2^-127 where bf16's
// least step makes that more; and code * step is exact in the 16-bit format the
// value came from: at most 7 significant bits, no larger than a, no finer than the format's
// least value (bf16: than 2^-126). The power of two makes the scaling exact in both
// directions, so codes do not depend on how they are computed. The scale byte is e + 127;
// 255 marks a block that held a NaN or an infinity, all of whose values come back NaN.
#pragma once

#include "mhc_device.h"

namespace mhc {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
constexpr uint32_t kCkptNan = 255;

// Larger of the magnitudes of each 16-bit half (as integers, which order like the values).
__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b)
{
    typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a),
                                                                  __builtin_bit_cast(u16x2_t, b)));
}
__device__ __forceinline__ uint32_t absmax_octet(u32x4 v)
{
    constexpr uint32_t kAbs = 0x7fff7fffu;
    return pk_max_u16(pk_max_u16(v[0] & kAbs, v[1] & kAbs), pk_max_u16(v[2] & kAbs, v[3] & kAbs));
}
// The other lanes' packed maxima: a pair of lanes (xor 1), then a quad (xor 2).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_pk_max(uint32_t m)
{
    return pk_max_u16(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, CTRL, 0xF, 0xF, true));
}
// A block's scale byte from its packed maximum.
template <bool H>
__device__ __forceinline__ uint32_t ckpt_scale(uint32_t pk)
{
    const uint32_t lo = pk & 0xffffu, hi = pk >> 16, a = lo > hi ? lo : hi;
    const uint32_t f = __float_as_uint(x16_lo<H>(a));
    const int s = (int)(f >> 23) - 6, least = H ? 103 : 1;
    return a >= (H ? 0x7c00u : 0x7f80u) ? kCkptNan : (uint32_t)(s > least ? s : least);
}
// Eight 16-bit values to eight codes. x * 2^-e is exact, and adding 1.5 * 2^23 rounds it to
// an integer (to nearest even) whose two's complement is the sum's low byte.
template <bool H>
__device__ __forceinline__ u32x2 ckpt_encode(u32x4 v, uint32_t scale)
{
    const float inv = __uint_as_float((254u - (scale == kCkptNan ? 127u : scale)) << 23);
    u32x2 out;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t w = v[2 * h + (e >> 1)];
            const float f = ((e & 1) ? x16_hi<H>(w) : x16_lo<H>(w)) * inv;
            r[e] = __float_as_uint(__builtin_amdgcn_fmed3f(f, -127.f, 127.f) + 12582912.f);
        }
        const uint32_t p01 = __builtin_amdgcn_perm(r[1], r[0], 0x0c0c0400u);
        const uint32_t p23 = __builtin_amdgcn_perm(r[3], r[2], 0x0c0c0400u);
        out[h] = scale == kCkptNan ? 0u : __builtin_amdgcn_perm(p23, p01, 0x05040100u);
    }
    return out;
}
// A scale byte's step (NaN for 255).
__device__ __forceinline__ float ckpt_step(uint32_t scale)
{
    return __uint_as_float(scale == kCkptNan ? 0x7fc00000u : scale << 23);
}
// Code e (0 .. 7) of an octet as a float.
__device__ __forceinline__ float ckpt_value(u32x2 c, int e, float step)
{
    return (float)(int)(int8_t)(c[e >> 2] >> (8 * (e & 3))) * step;
}
// Eight codes to eight 16-bit values (exact).
template <bool H>
__device__ __forceinline__ u32x4 ckpt_decode(u32x2 c, float step)
{
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float lo = ckpt_value(c, 2 * e, step), hi = ckpt_value(c, 2 * e + 1, step);
        v[e] = H ? pack_f16x2(lo, hi)
                 : __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
    }
    return v;
}

}  // namespace
}  // namespace mhc
