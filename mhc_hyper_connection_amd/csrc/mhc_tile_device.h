// mhc_tile_device.h -- what the tiled products share: direct loads to LDS with explicit waits, and
// the gated projections' activations.
#pragma once

#include "mhc_device.h"

namespace mhc {
namespace {

#define MHC_LDS __attribute__((address_space(3)))

// act(g) and act'(g). Past |g| = 64 both sigmoids are 0 or 1 to the last bit, and the
// derivative of z is taken at the clamped g, where it cannot overflow.
struct Act {
    float a, da;
};
template <int ACT>
__device__ __forceinline__ Act activation(float g)
{
#pragma clang fp contract(off)   // the same steps wherever it is inlined: h again is h
    constexpr float c = 1.5957691216057308f, q = 0.044715f;   // 2 sqrt(2 / pi)
    float z = g, dz = 1.f;
    if constexpr (ACT == 1) {
        const float gc = __builtin_amdgcn_fmed3f(g, -64.f, 64.f);
        z = c * fmaf(q * g * g, g, g);
        dz = fmaf(3.f * q * c * gc, gc, c);
    }
    const float s = __builtin_amdgcn_rcpf(1.f + __expf(-z));
    const float a = g * s;
    return {a, fmaf(a * (1.f - s), dz, s)};
}

// A raw buffer's descriptor as four words for the direct-to-LDS loads below: accesses at or
// past `bytes` write zeros.
__device__ __forceinline__ u32x4 descriptor(const void* base, uint32_t bytes)
{
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    return u32x4{(uint32_t)p, (uint32_t)(p >> 32) & 0xffffu, bytes, (uint32_t)kRsrcWord3};
}
// 64 lanes x 16 bytes from the buffer to LDS at `lds` (lane l to lds + 16 l). In inline
// assembly so that the compiler inserts no waits of its own before LDS reads; the kernel
// waits explicitly with the in-order vector memory counter. There is no register result. (The
// s_nop is the wait state that a write of m0 needs before its use as an LDS address.)
__device__ __forceinline__ void buffer_to_lds(u32x4 desc, uint32_t offset, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" : : "v"(offset), "s"(desc), "s"(lds) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads_and_barrier()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

}  // namespace
}  // namespace mhc
