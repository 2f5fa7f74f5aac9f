// mhc_mxfp4.hip -- gfx950 kernels of the microscaled 4-bit floats: 16-bit rows to codes and block
// scales, and back. The format and its arithmetic are in mhc_mxfp4_device.h.
//
// Both stream: per value 2 bytes against 17/32, and some two vector instructions. HBM bounds them: T = 16384, D = 7168
// (297 MB either way) 67 us there, 4.4 TB/s, and 50 back, 5.9 (a large copy moves 5.2). Small tensors take 2 to 3 us whatever is done.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "mhc_mxfp4_device.h"
#include "mhc_mxfp4_plan.h"

namespace mhc {
namespace mx {
namespace {

constexpr int kThr = 256;

// D a multiple of 128: rows have no padding and are one run of blocks. A thread takes 16 values (two
// lanes share a block) four times over.
constexpr int kUnits = 4;
template <bool H>
__global__ void __launch_bounds__(kThr)
quantise_flat_kernel(const uint16_t* __restrict__ x, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int64_t units)
{
    const int64_t u0 = (int64_t)blockIdx.x * (kThr * kUnits) + threadIdx.x;
    u32x4 v[kUnits][2];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        const int64_t u = u0 + k * kThr;
        const u32x4* p = reinterpret_cast<const u32x4*>(x) + 2 * (u < units ? u : units - 1);
        v[k][0] = p[0];
        v[k][1] = p[1];
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        const int64_t u = u0 + k * kThr;
        const uint32_t s = mx_scale<H>(mx_dpp_max<kQuadXor1>(mx_pk_max(mx_absmax(v[k][0]), mx_absmax(v[k][1]))));
        if (u < units) {
            reinterpret_cast<u32x2*>(codes)[u] = u32x2{mx_encode<H>(v[k][0], s), mx_encode<H>(v[k][1], s)};
            if (!(u & 1)) scales[u >> 1] = (uint8_t)s;
        }
    }
}

template <bool H>
__global__ void __launch_bounds__(kThr)
restore_flat_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, uint16_t* __restrict__ x, int64_t units)
{
    const int64_t u0 = (int64_t)blockIdx.x * (kThr * kUnits) + threadIdx.x;
    u32x2 c[kUnits];
    uint32_t s[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        const int64_t u = u0 + k * kThr, uc = u < units ? u : units - 1;
        c[k] = reinterpret_cast<const u32x2*>(codes)[uc];
        s[k] = scales[uc >> 1];
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        const int64_t u = u0 + k * kThr;
        if (u < units) {
            u32x4* p = reinterpret_cast<u32x4*>(x) + 2 * u;
            p[0] = mx_decode<H>(c[k][0], s[k]);
            p[1] = mx_decode<H>(c[k][1], s[k]);
        }
    }
}

// Any D: a thread to eight values of a row whose length is padded to whole words of scales (P octets), so
// that a quad of lanes shares a block. The padding's codes and scales are written as zeros.
// VEC: D is a multiple of 8, so that rows start on 16 bytes.
struct RowOctet {
    int64_t row;
    int o;
};
__device__ __forceinline__ RowOctet row_octet(int P)
{
    const int64_t first = (int64_t)blockIdx.x * kThr;
    const int64_t row0 = first / P;
    const uint32_t o = (uint32_t)(first - row0 * P) + threadIdx.x;
    const uint32_t dr = o / (uint32_t)P;
    return {row0 + dr, (int)(o - dr * (uint32_t)P)};
}

template <bool H, bool VEC>
__global__ void __launch_bounds__(kThr)
quantise_kernel(const uint16_t* __restrict__ x, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int64_t rows, int D, int P)
{
    const RowOctet at = row_octet(P);
    const bool live = at.row < rows;
    const int d = 8 * at.o;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (live && d < D) {
        const uint16_t* const p = x + at.row * D + d;
        if constexpr (VEC) v = *reinterpret_cast<const u32x4*>(p);
        else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (d + e < D) v[e / 2] |= (uint32_t)p[e] << (16 * (e & 1));
        }
    }
    const uint32_t s = mx_scale<H>(mx_dpp_max<kQuadXor2>(mx_dpp_max<kQuadXor1>(mx_absmax(v))));
    const int blocks = (D + kBlock - 1) / kBlock;
    if (live) {
        if (at.o < 4 * blocks) reinterpret_cast<uint32_t*>(codes)[at.row * (4 * blocks) + at.o] = mx_encode<H>(v, s);
        if (!(at.o & 3)) scales[at.row * (P / 4) + at.o / 4] = (uint8_t)(at.o < 4 * blocks ? s : 0u);
    }
}

template <bool H, bool VEC>
__global__ void __launch_bounds__(kThr)
restore_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, uint16_t* __restrict__ x, int64_t rows, int D, int P)
{
    const RowOctet at = row_octet(P);
    const int d = 8 * at.o;
    if (at.row >= rows || d >= D) return;
    const int blocks = (D + kBlock - 1) / kBlock;
    const u32x4 v = mx_decode<H>(reinterpret_cast<const uint32_t*>(codes)[at.row * (4 * blocks) + at.o], scales[at.row * (P / 4) + at.o / 4]);
    uint16_t* const p = x + at.row * D + d;
    if constexpr (VEC) *reinterpret_cast<u32x4*>(p) = v;
    else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (d + e < D) p[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
    }
}

unsigned flat_blocks(int64_t units) { return (unsigned)((units + kThr * kUnits - 1) / (kThr * kUnits)); }

template <bool H>
hipError_t quantise(int64_t rows, int D, const uint16_t* x, uint8_t* codes, uint8_t* scales, hipStream_t st)
{
    const int P = (int)scale_bytes(D) * 4;
    const dim3 grid((unsigned)octet_blocks(rows, D));
    if (D % 128 == 0) {
        const int64_t units = rows * (D / 16);
        hipLaunchKernelGGL(quantise_flat_kernel<H>, dim3(flat_blocks(units)), dim3(kThr), 0, st, x, codes, scales, units);
    } else if (D % 8 == 0) hipLaunchKernelGGL((quantise_kernel<H, true>), grid, dim3(kThr), 0, st, x, codes, scales, rows, D, P);
    else hipLaunchKernelGGL((quantise_kernel<H, false>), grid, dim3(kThr), 0, st, x, codes, scales, rows, D, P);
    return hipGetLastError();
}
template <bool H>
hipError_t restore(int64_t rows, int D, const uint8_t* codes, const uint8_t* scales, uint16_t* x, hipStream_t st)
{
    const int P = (int)scale_bytes(D) * 4;
    const dim3 grid((unsigned)octet_blocks(rows, D));
    if (D % 128 == 0) {
        const int64_t units = rows * (D / 16);
        hipLaunchKernelGGL(restore_flat_kernel<H>, dim3(flat_blocks(units)), dim3(kThr), 0, st, codes, scales, x, units);
    } else if (D % 8 == 0) hipLaunchKernelGGL((restore_kernel<H, true>), grid, dim3(kThr), 0, st, codes, scales, x, rows, D, P);
    else hipLaunchKernelGGL((restore_kernel<H, false>), grid, dim3(kThr), 0, st, codes, scales, x, rows, D, P);
    return hipGetLastError();
}

}  // namespace

int launch_quantise(int64_t rows, int D, const uint16_t* x, uint8_t* codes, uint8_t* scales, int x_f16, void* stream)
{
    clear_pending_error();
    hipStream_t st = (hipStream_t)stream;
    return (int)(x_f16 ? quantise<true>(rows, D, x, codes, scales, st) : quantise<false>(rows, D, x, codes, scales, st));
}

int launch_restore(int64_t rows, int D, const uint8_t* codes, const uint8_t* scales, uint16_t* x, int x_f16, void* stream)
{
    clear_pending_error();
    hipStream_t st = (hipStream_t)stream;
    return (int)(x_f16 ? restore<true>(rows, D, codes, scales, x, st) : restore<false>(rows, D, codes, scales, x, st));
}

}  // namespace mx
}  // namespace mhc
