// mhc_ckpt.hip -- gfx950 kernels of the 8-bit checkpoints: 16-bit rows to codes and block
// scales, and back, and hc_post with its output's checkpoint written beside it. The format
// and its arithmetic are in mhc_ckpt_device.h.
//
// All three stream: per value 2 bytes against 1 + 1/32, some ten vector instructions.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "mhc_ckpt_device.h"
#include "mhc_train_plan.h"

namespace mhc {
namespace {

constexpr int kThr = 256;

// Thread -> (row, octet) of rows whose last block is padded to a whole one (P = 4 ceil(D / 32)
// octets), so that the four lanes of a quad always share a block. The workgroup's first
// index is split once in 64 bits, the lane's offset from it in 32.
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

// D a multiple of 32: the rows are one run of blocks. A thread takes 16 values (two lanes
// share a block) four times over.
constexpr int kUnits = 4;
template <bool H>
__global__ void __launch_bounds__(kThr)
checkpoint_flat_kernel(const uint16_t* __restrict__ x, int8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                       int64_t units)
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
        const uint32_t m = dpp_pk_max<kQuadXor1>(pk_max_u16(absmax_octet(v[k][0]), absmax_octet(v[k][1])));
        const uint32_t s = ckpt_scale<H>(m);
        const u32x2 a = ckpt_encode<H>(v[k][0], s), b = ckpt_encode<H>(v[k][1], s);
        if (u < units) {
            reinterpret_cast<u32x4*>(codes)[u] = u32x4{a[0], a[1], b[0], b[1]};
            if (!(u & 1)) scales[u >> 1] = (uint8_t)s;
        }
    }
}

template <bool H>
__global__ void __launch_bounds__(kThr)
checkpoint_kernel(const uint16_t* __restrict__ x, int8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                  int64_t rows, int D, int P)
{
    const RowOctet at = row_octet(P);
    const bool live = at.row < rows && at.o < D / 8;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (live) v = *reinterpret_cast<const u32x4*>(x + at.row * D + 8 * at.o);
    const uint32_t s = ckpt_scale<H>(dpp_pk_max<kQuadXor2>(dpp_pk_max<kQuadXor1>(absmax_octet(v))));
    if (live) {
        *reinterpret_cast<u32x2*>(codes + at.row * D + 8 * at.o) = ckpt_encode<H>(v, s);
        if (!(at.o & 3)) scales[at.row * (P / 4) + at.o / 4] = (uint8_t)s;
    }
}

template <bool H>
__global__ void __launch_bounds__(kThr)
restore_flat_kernel(const int8_t* __restrict__ codes, const uint8_t* __restrict__ scales, uint16_t* __restrict__ x,
                    int64_t units)
{
    const int64_t u0 = (int64_t)blockIdx.x * (kThr * kUnits) + threadIdx.x;
    u32x4 c[kUnits];
    uint32_t s[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        const int64_t u = u0 + k * kThr, uc = u < units ? u : units - 1;
        c[k] = reinterpret_cast<const u32x4*>(codes)[uc];
        s[k] = scales[uc >> 1];
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        const int64_t u = u0 + k * kThr;
        const float step = ckpt_step(s[k]);
        if (u < units) {
            u32x4* p = reinterpret_cast<u32x4*>(x) + 2 * u;
            p[0] = ckpt_decode<H>(u32x2{c[k][0], c[k][1]}, step);
            p[1] = ckpt_decode<H>(u32x2{c[k][2], c[k][3]}, step);
        }
    }
}

template <bool H>
__global__ void __launch_bounds__(kThr)
restore_kernel(const int8_t* __restrict__ codes, const uint8_t* __restrict__ scales, uint16_t* __restrict__ x,
               int64_t rows, int D, int P)
{
    const RowOctet at = row_octet(P);
    if (at.row >= rows || at.o >= D / 8) return;
    const u32x2 c = *reinterpret_cast<const u32x2*>(codes + at.row * D + 8 * at.o);
    const float step = ckpt_step(scales[at.row * (P / 4) + at.o / 4]);
    *reinterpret_cast<u32x4*>(x + at.row * D + 8 * at.o) = ckpt_decode<H>(c, step);
}

// hc_post (mhc_post.hip's arithmetic, term for term, so that `out` has the same bits) with
// the checkpoint of each output stream made from the rounded values in registers: the
// streams are not read again.
template <int N, bool H>
__global__ void __launch_bounds__(kThr)
post_checkpoint_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ residual,
                       const float* __restrict__ post, const float* __restrict__ comb, uint16_t* __restrict__ out,
                       int8_t* __restrict__ codes, uint8_t* __restrict__ scales, int64_t T, int D, int P)
{
    const RowOctet at = row_octet(P);
    const bool live = at.row < T && at.o < D / 8;
    const int64_t t = at.row < T ? at.row : T - 1;   // the padding lanes compute along from the
    const int d = 8 * (at.o < D / 8 ? at.o : 0);      // row's first octet and store nothing
    const u32x4 xv = *reinterpret_cast<const u32x4*>(x + t * (int64_t)D + d);
    u32x4 rv[N];
#pragma unroll
    for (int i = 0; i < N; ++i) rv[i] = *reinterpret_cast<const u32x4*>(residual + (t * N + i) * (int64_t)D + d);
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float p = post[t * N + j];
        float c[N];
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] = comb[(t * N + i) * N + j];
        float acc[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            acc[2 * e] = p * x16_lo<H>(xv[e]);
            acc[2 * e + 1] = p * x16_hi<H>(xv[e]);
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                acc[2 * e] = fmaf(c[i], x16_lo<H>(rv[i][e]), acc[2 * e]);
                acc[2 * e + 1] = fmaf(c[i], x16_hi<H>(rv[i][e]), acc[2 * e + 1]);
            }
        u32x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = live ? pack_x16<H>(acc[2 * e], acc[2 * e + 1]) : 0u;
        const uint32_t s = ckpt_scale<H>(dpp_pk_max<kQuadXor2>(dpp_pk_max<kQuadXor1>(absmax_octet(o))));
        if (live) {
            const int64_t row = t * N + j;
            __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(out + row * D + d));
            __builtin_nontemporal_store(ckpt_encode<H>(o, s), reinterpret_cast<u32x2*>(codes + row * D + d));
            if (!(at.o & 3)) scales[row * (P / 4) + at.o / 4] = (uint8_t)s;
        }
    }
}

unsigned flat_blocks(int64_t units) { return (unsigned)((units + kThr * kUnits - 1) / (kThr * kUnits)); }

}  // namespace

int launch_checkpoint(int64_t rows, int D, const uint16_t* x, int8_t* codes, uint8_t* scales, int x_f16, void* stream)
{
    clear_pending_error();
    hipStream_t st = (hipStream_t)stream;
    if (D % kCkptBlock == 0) {
        const int64_t units = rows * (D / 16);
        if (x_f16) hipLaunchKernelGGL(checkpoint_flat_kernel<true>, dim3(flat_blocks(units)), dim3(kThr), 0, st, x, codes, scales, units);
        else hipLaunchKernelGGL(checkpoint_flat_kernel<false>, dim3(flat_blocks(units)), dim3(kThr), 0, st, x, codes, scales, units);
    } else {
        const dim3 grid((unsigned)octet_blocks(rows, D));
        const int P = ckpt_octets(D);
        if (x_f16) hipLaunchKernelGGL(checkpoint_kernel<true>, grid, dim3(kThr), 0, st, x, codes, scales, rows, D, P);
        else hipLaunchKernelGGL(checkpoint_kernel<false>, grid, dim3(kThr), 0, st, x, codes, scales, rows, D, P);
    }
    return (int)hipGetLastError();
}

int launch_checkpoint_restore(int64_t rows, int D, const int8_t* codes, const uint8_t* scales, uint16_t* x, int x_f16,
                              void* stream)
{
    clear_pending_error();
    hipStream_t st = (hipStream_t)stream;
    if (D % kCkptBlock == 0) {
        const int64_t units = rows * (D / 16);
        if (x_f16) hipLaunchKernelGGL(restore_flat_kernel<true>, dim3(flat_blocks(units)), dim3(kThr), 0, st, codes, scales, x, units);
        else hipLaunchKernelGGL(restore_flat_kernel<false>, dim3(flat_blocks(units)), dim3(kThr), 0, st, codes, scales, x, units);
    } else {
        const dim3 grid((unsigned)octet_blocks(rows, D));
        const int P = ckpt_octets(D);
        if (x_f16) hipLaunchKernelGGL(restore_kernel<true>, grid, dim3(kThr), 0, st, codes, scales, x, rows, D, P);
        else hipLaunchKernelGGL(restore_kernel<false>, grid, dim3(kThr), 0, st, codes, scales, x, rows, D, P);
    }
    return (int)hipGetLastError();
}

int launch_post_checkpoint(int64_t T, int n, int D, const uint16_t* x, const uint16_t* residual, const float* post,
                           const float* comb, uint16_t* out, int8_t* codes, uint8_t* scales, int x_f16, void* stream)
{
    clear_pending_error();
    hipStream_t st = (hipStream_t)stream;
    const dim3 grid((unsigned)octet_blocks(T, D));
    const int P = ckpt_octets(D);
#define MHC_POSTC(NV, HV) hipLaunchKernelGGL((post_checkpoint_kernel<NV, HV>), grid, dim3(kThr), 0, st, x, residual, post, comb, out, codes, scales, T, D, P)
    if (n == 4 && !x_f16) MHC_POSTC(4, false);
    else if (n == 6 && !x_f16) MHC_POSTC(6, false);
    else if (n == 8 && !x_f16) MHC_POSTC(8, false);
    else if (n == 4) MHC_POSTC(4, true);
    else if (n == 6) MHC_POSTC(6, true);
    else if (n == 8) MHC_POSTC(8, true);
    else return (int)hipErrorInvalidValue;
#undef MHC_POSTC
    return (int)hipGetLastError();
}

}  // namespace mhc
