// mhc_post_bwd.hip -- gfx950 kernel of hc_post's backward. With hc_post as mhc_post.hip
// computes it,
//     out[t][j][d] = post[t][j] x[t][d] + sum_i comb[t][i][j] residual[t][i][d],
// and G = dL/dout, per token:
//     gradX[d]           = sum_j post[j] G[j][d]
//     gradResidual[i][d] = sum_j comb[i][j] G[j][d]
//     gradPost[j]        = sum_d G[j][d] x[d]
//     gradComb[i][j]     = sum_d residual[i][d] G[j][d]
// One pass: a lane holds the n streams of G at an octet of positions, forms both mixed
// gradients from it and adds its products with x and the residual streams to n + n*n sums,
// which the token's lanes join at the end. x and the residual streams only enter the sums,
// so either may come as an 8-bit checkpoint, decoded in registers.
//
// Memory-bound: per token 2nD (G) + 2(n + 1)D (or 33/32 (n + 1)D) read, 2(n + 1)D written. At
// T = 16384, n = 4, D = 7168 from checkpoints 515 us, 5.3 TB/s (a large copy: 5.2).
//
// Four waves a token where each then still has a few octets a lane for the n + n*n sums
// that it joins at the end (D >= 512 n), and for few tokens, which would leave the chip empty;
// else one. Measured from checkpoints, T = 16384: n = 4, D = 7168 515 us against 535 with one
// wave, D = 2048 133 against 148, D = 512 58 against 32; n = 6, D = 2048 214 against 212;
// T = 512: n = 8, D = 7168 38 against 59.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "mhc_ckpt_device.h"
#include "mhc_train_plan.h"

namespace mhc {
namespace {

constexpr int kThr = 256;

// An octet of 16-bit values, or of codes with their step.
template <bool H, bool Q> struct Octet;
template <bool H> struct Octet<H, false> {
    u32x4 v;
    __device__ __forceinline__ void load(const uint16_t* p, const int8_t*, const uint8_t*, int64_t at, int64_t, int)
    {
        v = *reinterpret_cast<const u32x4*>(p + at);
    }
    __device__ __forceinline__ float get(int e) const { return (e & 1) ? x16_hi<H>(v[e >> 1]) : x16_lo<H>(v[e >> 1]); }
};
template <bool H> struct Octet<H, true> {
    u32x2 c;
    uint32_t s;
    __device__ __forceinline__ void load(const uint16_t*, const int8_t* codes, const uint8_t* scales, int64_t at,
                                         int64_t row_scales, int o)
    {
        c = *reinterpret_cast<const u32x2*>(codes + at);
        s = scales[row_scales + (o >> 2)];
    }
    __device__ __forceinline__ float get(int e) const { return ckpt_value(c, e, ckpt_step(s)); }
};

// Sum over the wave's 64 lanes, in a fixed order; every lane gets it.
__device__ __forceinline__ float wave_sum(float v)
{
    v += dpp<kQuadXor1>(v);
    v += dpp<kQuadXor2>(v);
    v += dpp<kRowRor4>(v);
    v += dpp<kRowRor8>(v);
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    return v;
}

// W waves per token, 4 / W tokens per workgroup.
template <int N, bool H, bool QX, bool QR>
__global__ void __launch_bounds__(kThr, N == 8 ? (H ? 3 : 2) : 4 - N / 6)
post_bwd_kernel(PostBwdArgs a, int64_t T, int D, int NB, int W)
{
    constexpr int V = N + N * N;
    __shared__ float red[4][V];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t t = W == 1 ? (int64_t)blockIdx.x * 4 + wave : (int64_t)blockIdx.x;
    const bool live = t < T;
    const int64_t tt = live ? t : T - 1;
    float post[N], comb[N][N], sp[N], sc[N][N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        post[j] = a.post[tt * N + j];
        sp[j] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) {
            comb[i][j] = a.comb[(tt * N + i) * N + j];
            sc[i][j] = 0.f;
        }
    const int octets = live ? D / 8 : 0;
    for (int o = lane + (W == 1 ? 0 : 64 * wave); o < octets; o += 64 * W) {
        u32x4 gv[N];
        Octet<H, QR> rv[N];
        Octet<H, QX> xv;
#pragma unroll
        for (int j = 0; j < N; ++j)
            gv[j] = *reinterpret_cast<const u32x4*>(a.grad_out + (tt * N + j) * (int64_t)D + 8 * o);
#pragma unroll
        for (int i = 0; i < N; ++i)
            rv[i].load(a.residual, a.r_codes, a.r_scales, (tt * N + i) * (int64_t)D + 8 * o, (tt * N + i) * (int64_t)NB, o);
        xv.load(a.x, a.x_codes, a.x_scales, tt * (int64_t)D + 8 * o, tt * (int64_t)NB, o);
        float g[N][8];
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) g[j][e] = (e & 1) ? x16_hi<H>(gv[j][e >> 1]) : x16_lo<H>(gv[j][e >> 1]);
        float acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float xe = xv.get(e);
            acc[e] = post[0] * g[0][e];
            sp[0] = fmaf(g[0][e], xe, sp[0]);
#pragma unroll
            for (int j = 1; j < N; ++j) {
                acc[e] = fmaf(post[j], g[j][e], acc[e]);
                sp[j] = fmaf(g[j][e], xe, sp[j]);
            }
        }
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pack_x16<H>(acc[2 * e], acc[2 * e + 1]);
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(a.grad_x + tt * (int64_t)D + 8 * o));
#pragma unroll
        for (int i = 0; i < N; ++i) {
            __builtin_amdgcn_sched_barrier(0);   // one stream's values decoded at a time, not all at once
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float re = rv[i].get(e);
                acc[e] = comb[i][0] * g[0][e];
                sc[i][0] = fmaf(g[0][e], re, sc[i][0]);
#pragma unroll
                for (int j = 1; j < N; ++j) {
                    acc[e] = fmaf(comb[i][j], g[j][e], acc[e]);
                    sc[i][j] = fmaf(g[j][e], re, sc[i][j]);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = pack_x16<H>(acc[2 * e], acc[2 * e + 1]);
            __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(a.grad_residual + (tt * N + i) * (int64_t)D + 8 * o));
        }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float v = wave_sum(sp[j]);
        if (lane == 0) red[wave][j] = v;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float v = wave_sum(sc[i][j]);
            if (lane == 0) red[wave][N + i * N + j] = v;
        }
    __syncthreads();
    if (W == 1) {
        for (int k = lane; k < V && live; k += 64) {
            const float v = red[wave][k];
            if (k < N) a.grad_post[t * N + k] = v;
            else a.grad_comb[t * N * N + (k - N)] = v;
        }
    } else if (threadIdx.x < V) {
        const int k = threadIdx.x;
        const float v = (red[0][k] + red[1][k]) + (red[2][k] + red[3][k]);
        if (k < N) a.grad_post[t * N + k] = v;
        else a.grad_comb[t * N * N + (k - N)] = v;
    }
}

template <int N, bool H>
hipError_t launch(int64_t T, int D, PostBwdArgs a, hipStream_t st)
{
    const int W = post_bwd_waves(T, N, D), NB = ckpt_blocks(D);
    const int64_t most = post_bwd_launch_tokens(W);
    for (; T > 0; T -= most) {
        const int64_t Tc = T < most ? T : most;
        const dim3 grid((unsigned)post_bwd_blocks(Tc, W));
        if (a.x && a.residual) hipLaunchKernelGGL((post_bwd_kernel<N, H, false, false>), grid, dim3(kThr), 0, st, a, Tc, D, NB, W);
        else if (a.residual) hipLaunchKernelGGL((post_bwd_kernel<N, H, true, false>), grid, dim3(kThr), 0, st, a, Tc, D, NB, W);
        else if (a.x) hipLaunchKernelGGL((post_bwd_kernel<N, H, false, true>), grid, dim3(kThr), 0, st, a, Tc, D, NB, W);
        else hipLaunchKernelGGL((post_bwd_kernel<N, H, true, true>), grid, dim3(kThr), 0, st, a, Tc, D, NB, W);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        if (T > most) a = post_bwd_after(a, Tc, N, D);
    }
    return hipSuccess;
}

}  // namespace

int launch_post_backward(int64_t T, int n, int D, const PostBwdArgs& a, int x_f16, void* stream)
{
    clear_pending_error();
    hipStream_t st = (hipStream_t)stream;
    if (n == 4) return (int)(x_f16 ? launch<4, true>(T, D, a, st) : launch<4, false>(T, D, a, st));
    if (n == 6) return (int)(x_f16 ? launch<6, true>(T, D, a, st) : launch<6, false>(T, D, a, st));
    if (n == 8) return (int)(x_f16 ? launch<8, true>(T, D, a, st) : launch<8, false>(T, D, a, st));
    return (int)hipErrorInvalidValue;
}

}  // namespace mhc
