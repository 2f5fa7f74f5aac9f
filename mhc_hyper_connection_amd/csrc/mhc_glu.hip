// mhc_glu.hip -- gfx950 kernels of the gated projection and its backward.
//
//   forward   g = x Wg^T, u = x Wu^T, h = act(g) (.) u
//   backward  with dh = dL/dh: g and u again, dg = dh u act'(g), du = dh act(g), h = act(g) u,
//             dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x
// x [T, D], Wg and Wu [F, D], h and dh [T, F], bf16 or fp16 (template flag H); act(g) =
// g sigmoid(z) with z = g (SiLU) or 2 sqrt(2/pi) (g + 0.044715 g^3) (GELU's tanh form).
// Products accumulate in fp32 on the matrix cores; g, u and the activation stay in fp32
// registers; dg and du are rounded once to the 16-bit format (they are the operands of the next
// products), and so is each result.
//
// Four products share one tiled kernel (tile_kernel): C = A B over a reduction of kBK = 32
// positions per stage. The operand whose rows become C's rows is always the one whose
// index is contiguous in the result, so that a lane of the matrix-core result (4 consecutive
// rows of one column) holds consecutive results.
//   kForward, kRecompute  rows: Wg and Wu side by side (a wave holds g and u of the same f);
//                         columns: tokens; both operands contiguous along the reduction
//   kGradX                rows: d, columns: tokens; W is contiguous across the reduction
//   kGradW                rows: d, columns: f; both contiguous across the reduction
// An operand contiguous across the reduction is read from LDS by the transposing read
// (ds_read_b64_tr_b16: lane i of 16 gets column i of the 4 x 16 block that the 16 lanes
// address), so that nothing is transposed in memory.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "mhc_device.h"
#include "mhc_glu_plan.h"

namespace mhc {
namespace glu {
namespace {

enum Mode { kForward, kRecompute, kGradX, kGradW };

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
#define MHC_LDS __attribute__((address_space(3)))

template <bool H>
__device__ __forceinline__ f32x4 mfma(s16x8 a, s16x8 b, f32x4 c)
{
    if constexpr (H) return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// act(g) and act'(g). Past |g| = 64 both sigmoids are 0 or 1 to the last bit, and the
// derivative of z is taken at the clamped g, where it cannot overflow.
struct Act {
    float a, da;
};
__device__ __forceinline__ Act activation(float g, int act)
{
    constexpr float c = 1.5957691216057308f, q = 0.044715f;   // 2 sqrt(2 / pi)
    float z = g, dz = 1.f;
    if (act) {
        const float gc = fminf(fmaxf(g, -64.f), 64.f);
        z = c * (g + q * g * g * g);
        dz = c * (1.f + 3.f * q * gc * gc);
    }
    const float s = __builtin_amdgcn_rcpf(1.f + __expf(-z));
    const float a = g * s;
    return {a, s + a * (1.f - s) * dz};
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

// Workgroup -> tile. Workgroups b, b + 8, .. run on one XCD; each XCD takes a contiguous
// run of the tile order, which walks the columns of kGroup rows of tiles before the next
// rows: the tiles in flight on an XCD then share kGroup row operands and a few column
// operands in its L2.
constexpr int kGroup = 4;
__device__ __forceinline__ bool tile_of(int64_t na, int64_t nb, int64_t* a, int64_t* b)
{
    const int64_t total = na * nb, per = (total + 7) / 8;
    const int64_t t = (int64_t)(blockIdx.x % 8) * per + blockIdx.x / 8;
    if (blockIdx.x / 8 >= per || t >= total) return false;
    const int64_t group = t / (kGroup * nb), r = t - group * kGroup * nb;
    const int64_t rows = na - group * kGroup < kGroup ? na - group * kGroup : kGroup;
    *a = group * kGroup + r % rows;
    *b = r / rows;
    return true;
}

struct TileArgs {
    Args t;
    int64_t T;
    int D, F, act;
    int64_t na, nb;
    int64_t steps, per;   // stages in all, stages of a part
    float* part;          // NULL, or the parts' sums [split][...] in fp32
};

// WA x WB waves of IA x IB 16 x 16 results each. LDS: a ring of 4 stages of both operands.
// At step k a wave waits for its own loads of stage k, meets the others (whose reads of
// stage k - 1 are then done as well), sends off the loads of stage k + 3 into the slot of stage k - 1
// and multiplies stage k. Loads past the end of the reduction bring zeros.
template <int MODE, bool H, int WA, int WB, int IA, int IB>
__global__ void __launch_bounds__(64 * WA * WB, 2)
tile_kernel(TileArgs p)
{
    constexpr int NW = WA * WB;
    constexpr int AR = 16 * WA * IA, BC = 16 * WB * IB;          // rows and columns of the tile
    constexpr int ASZ = AR * 2 * kBK, BSZ = BC * 2 * kBK;        // bytes of a stage
    constexpr int QA = AR / 16 / NW, QB = BC / 16 / NW;          // direct loads of a wave per stage
    constexpr int R = 4;
    constexpr bool A_ACROSS = MODE == kGradX || MODE == kGradW;  // A contiguous across the reduction
    constexpr bool B_ACROSS = MODE == kGradW;
    constexpr bool GATED = MODE == kForward || MODE == kRecompute;
    static_assert(QA * 16 * NW == AR && QB * 16 * NW == BC, "whole direct loads");
    static_assert(!GATED || QA % 2 == 0, "a direct load is of one of the two weights");
    __shared__ __attribute__((aligned(1024))) char lds[R * (ASZ + BSZ)];

    int64_t ta, tb;
    if (!tile_of(p.na, p.nb, &ta, &tb)) return;   // the padding of the last run of tiles
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wa = wave / WB, wb = wave % WB;
    const int j = lane & 15, kg = lane >> 4;
    const int D = p.D, F = p.F;
    const int64_t T = p.T;
    const int half_steps = (F + kBK - 1) / kBK;                  // kGradX: stages of either weight
    // kGradW: the tiles of Wg's gradient, then those of Wu's
    const int64_t nbh = MODE == kGradW ? p.nb / 2 : p.nb;
    const int up = MODE == kGradW && tb >= nbh ? 1 : 0;
    const int64_t a0 = ta * (GATED ? AR / 2 : AR);               // first f (gated) or d
    const int64_t b0 = (tb - up * nbh) * BC;                     // first token, or f

    const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>(lds));
    const uint32_t ldsb = lds0 + R * ASZ;

    // --- loads. Contiguous along the reduction: LDS rows of 64 bytes, a load is 16 rows; the 16-byte
    // chunk c of row r sits at c ^ s(r), with s so that the 16 rows of an operand read meet
    // all banks: s = (r / 4) % 4 for 16 rows in a run, (r / 8) % 4 for the gated rows, which
    // are read 4 of every 8. Across: rows of one reduction position, chunk c of row k at
    // c ^ 2 ((k % 4) + 4 ((k / 8) % 2)).
    constexpr int CA = AR / 8, CB = BC / 8;                      // chunks of an across row
    uint32_t va[QA], vb[QB];
    int ka[QA], kb[QB];                                          // the chunk's place in the stage (along)
#pragma unroll
    for (int q = 0; q < QA; ++q) {
        const int i = wave + NW * q;                             // the load's number in the stage
        if constexpr (A_ACROSS) {
            const int k = i * (64 / CA) + lane / CA, c = (lane % CA) ^ (2 * ((k & 3) + 4 * ((k >> 3) & 1)));
            va[q] = (uint32_t)((int64_t)k * D * 2) + (uint32_t)(a0 + 8 * c) * 2;
            ka[q] = 0;
        } else {
            const int r = 16 * i + lane / 4, c = (lane & 3) ^ ((r >> 3) & 3);
            va[q] = (uint32_t)(r % (AR / 2)) * (uint32_t)D * 2 + 16 * c;
            ka[q] = 8 * c;
        }
    }
#pragma unroll
    for (int q = 0; q < QB; ++q) {
        const int i = wave + NW * q;
        if constexpr (B_ACROSS) {
            const int k = i * (64 / CB) + lane / CB, c = (lane % CB) ^ (2 * ((k & 3) + 4 * ((k >> 3) & 1)));
            vb[q] = (uint32_t)k * (uint32_t)F * 4 + (uint32_t)((int64_t)up * F + b0 + 8 * c) * 2;
            kb[q] = 0;
        } else {
            const int r = 16 * i + lane / 4, c = (lane & 3) ^ ((r >> 2) & 3);
            vb[q] = (uint32_t)r * (uint32_t)(MODE == kGradX ? 2 * F : D) * 2 + 16 * c;
            kb[q] = 8 * c;
        }
    }
    const int64_t brow = !B_ACROSS ? (T - b0 < BC ? T - b0 : BC) : 0;   // rows of B that exist
    const int64_t arow = GATED ? (F - a0 < AR / 2 ? F - a0 : AR / 2) : 0;
    u32x4 dag, dau, db;
    if constexpr (GATED) {
        dag = descriptor(p.t.w_gate + a0 * D, (uint32_t)(arow * D * 2));
        dau = descriptor(p.t.w_up + a0 * D, (uint32_t)(arow * D * 2));
        db = descriptor(p.t.x + b0 * D, (uint32_t)(brow * D * 2));
    } else if constexpr (MODE == kGradX) {
        db = descriptor(p.t.dgu + b0 * 2 * F, (uint32_t)(brow * 2 * F * 2));
    }
    auto rows_left = [](int64_t n, int64_t k) { return (uint32_t)(n - k <= 0 ? 0 : (n - k < kBK ? n - k : kBK)); };
    auto issue = [&](int64_t step, int slot) __attribute__((always_inline)) {
        const uint32_t la = lds0 + slot * ASZ + wave * 1024, lb = ldsb + slot * BSZ + wave * 1024;
        if constexpr (GATED) {
            const int k = (int)(step * kBK);
#pragma unroll
            for (int q = 0; q < QA; ++q)
                buffer_to_lds(q < QA / 2 ? dag : dau, k + ka[q] < D ? va[q] + 2 * k : kOutOfRange, la + q * NW * 1024);
#pragma unroll
            for (int q = 0; q < QB; ++q)
                buffer_to_lds(db, k + kb[q] < D ? vb[q] + 2 * k : kOutOfRange, lb + q * NW * 1024);
        } else if constexpr (MODE == kGradX) {
            const int hf = step >= half_steps ? 1 : 0;
            const int64_t k = (step - (int64_t)hf * half_steps) * kBK;
            const uint32_t left = rows_left(F, k);
            const u32x4 da = descriptor((hf ? p.t.w_up : p.t.w_gate) + k * D, left * (uint32_t)D * 2);
#pragma unroll
            for (int q = 0; q < QA; ++q) buffer_to_lds(da, va[q], la + q * NW * 1024);
#pragma unroll
            for (int q = 0; q < QB; ++q)
                buffer_to_lds(db, k + kb[q] < F ? vb[q] + (uint32_t)(2 * (k + (int64_t)hf * F)) : kOutOfRange, lb + q * NW * 1024);
        } else {
            const int64_t k = step * kBK;
            const uint32_t left = rows_left(T, k);
            const u32x4 da = descriptor(p.t.x + (left ? k : 0) * D, left * (uint32_t)D * 2);
            const u32x4 dd = descriptor(p.t.dgu + (left ? k : 0) * 2 * F, left * (uint32_t)F * 4);
#pragma unroll
            for (int q = 0; q < QA; ++q) buffer_to_lds(da, va[q], la + q * NW * 1024);
#pragma unroll
            for (int q = 0; q < QB; ++q) buffer_to_lds(dd, vb[q], lb + q * NW * 1024);
        }
    };

    // --- operand reads. Along: lane (j, kg) takes chunk kg of row j; the gated rows of a
    // pair of results (h = 0, 1) are 8 (j / 4) + 4 h + j % 4, so that a lane's two results
    // are 8 consecutive f.
    const uint32_t aoff = A_ACROSS ? (uint32_t)((8 * kg + (j >> 2)) * (AR * 2) +
                                                (((IA * 2 * wa + ((j & 3) >> 1)) ^ (2 * ((j >> 2) + 4 * (kg & 1)))) << 4) + (j & 1) * 8)
                                   : (uint32_t)((16 * wa * IA / 2 + 8 * (j >> 2) + (j & 3)) * 64 + ((kg ^ (j >> 2)) << 4));
    const uint32_t boff = B_ACROSS ? (uint32_t)((8 * kg + (j >> 2)) * (BC * 2) +
                                                (((IB * 2 * wb + ((j & 3) >> 1)) ^ (2 * ((j >> 2) + 4 * (kg & 1)))) << 4) + (j & 1) * 8)
                                   : (uint32_t)((16 * wb * IB + j) * 64 + ((kg ^ (j >> 2)) << 4));
    auto read_along = [](uint32_t at) { return *(const MHC_LDS s16x8*)(uintptr_t)at; };
    auto read_across = [](uint32_t at, int row_bytes) {
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MHC_LDS s16x4*)(uintptr_t)at);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MHC_LDS s16x4*)(uintptr_t)(at + 4 * row_bytes));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };

    f32x4 acc[IA][IB];
#pragma unroll
    for (int i = 0; i < IA; ++i)
#pragma unroll
        for (int q = 0; q < IB; ++q) acc[i][q] = f32x4{0.f, 0.f, 0.f, 0.f};

    auto multiply = [&](int slot) __attribute__((always_inline)) {
        const uint32_t la = lds0 + slot * ASZ, lb = ldsb + slot * BSZ;
        s16x8 bf[IB];
#pragma unroll
        for (int q = 0; q < IB; ++q) {
            if constexpr (B_ACROSS) bf[q] = read_across(lb + (boff ^ (q << 5)), BC * 2);
            else bf[q] = read_along(lb + boff + q * 1024);
        }
#pragma unroll
        for (int i = 0; i < IA; ++i) {
            s16x8 af;
            if constexpr (A_ACROSS) af = read_across(la + (aoff ^ (i << 5)), AR * 2);
            else {   // gated: results 0 .. IA/2 - 1 are the gate's, the rest the up projection's
                const int i2 = i % (IA / 2);
                af = read_along(la + aoff + (i < IA / 2 ? 0 : AR / 2 * 64) + (i2 / 2) * 2048 + (i2 % 2) * 256);
            }
#pragma unroll
            for (int q = 0; q < IB; ++q) acc[i][q] = mfma<H>(af, bf[q], acc[i][q]);
        }
    };

    const int64_t k0 = (int64_t)blockIdx.y * p.per, k1 = k0 + p.per < p.steps ? k0 + p.per : p.steps;
    issue(k0, 0);
    issue(k0 + 1, 1);
    issue(k0 + 2, 2);
    for (int64_t k = k0; k < k1; k += R) {
#pragma unroll
        for (int s = 0; s < R; ++s) {
            if (k + s < k1) {
                wait_loads_and_barrier<2 * (QA + QB)>();
                issue(k + s + 3, (s + 3) % R);
                multiply(s);
            }
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");   // no load is left behind in LDS at the end

    // --- results: lane (j, kg) holds rows 4 kg .. 4 kg + 3 of column j of each 16 x 16 block
    if constexpr (GATED) {
#pragma unroll
        for (int q = 0; q < IB; ++q) {
            const int64_t t = b0 + 16 * (wb * IB + q) + j;
#pragma unroll
            for (int i = 0; i < IA / 4; ++i) {
                const int64_t f = a0 + 16 * wa * IA / 2 + 32 * i + 8 * kg;
                if (t < T && f < F) {
                    u32x4 dh = {0u, 0u, 0u, 0u};
                    if constexpr (MODE == kRecompute) dh = *reinterpret_cast<const u32x4*>(p.t.grad_h + t * F + f);
                    u32x4 hv, gv, uv;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float hh[2], dg[2], du[2];
#pragma unroll
                        for (int l = 0; l < 2; ++l) {
                            const int r = 2 * e + l;                            // f + r
                            const float gg = acc[2 * i + r / 4][q][r % 4], uu = acc[IA / 2 + 2 * i + r / 4][q][r % 4];
                            const Act ac = activation(gg, p.act);
                            const float d = l ? x16_hi<H>(dh[e]) : x16_lo<H>(dh[e]);
                            hh[l] = ac.a * uu;
                            dg[l] = d * uu * ac.da;
                            du[l] = d * ac.a;
                        }
                        hv[e] = pack_x16<H>(hh[0], hh[1]);
                        gv[e] = pack_x16<H>(dg[0], dg[1]);
                        uv[e] = pack_x16<H>(du[0], du[1]);
                    }
                    if (MODE == kForward || p.t.h) *reinterpret_cast<u32x4*>(p.t.h + t * F + f) = hv;
                    if constexpr (MODE == kRecompute) {
                        *reinterpret_cast<u32x4*>(p.t.dgu + t * 2 * F + f) = gv;
                        *reinterpret_cast<u32x4*>(p.t.dgu + t * 2 * F + F + f) = uv;
                    }
                }
            }
        }
    } else {
        // [column][row], rows contiguous: grad_x [T][D], or a weight's gradient [F][D]
        const int64_t ncol = MODE == kGradX ? T : F;
        uint16_t* const out = MODE == kGradX ? p.t.grad_x : (up ? p.t.grad_w_up : p.t.grad_w_gate);
        float* const part = p.part ? p.part + ((int64_t)blockIdx.y * (MODE == kGradX ? T : 2 * (int64_t)F) + (int64_t)up * F) * D : nullptr;
#pragma unroll
        for (int q = 0; q < IB; ++q) {
            const int64_t c = b0 + 16 * (wb * IB + q) + j;
#pragma unroll
            for (int i = 0; i < IA; ++i) {
                const int64_t d = a0 + 16 * (wa * IA + i) + 4 * kg;
                if (c < ncol && d < D) {
                    if (part) *reinterpret_cast<f32x4*>(part + c * D + d) = acc[i][q];
                    else *reinterpret_cast<u32x2*>(out + c * D + d) = u32x2{pack_x16<H>(acc[i][q][0], acc[i][q][1]), pack_x16<H>(acc[i][q][2], acc[i][q][3])};
                }
            }
        }
    }
}

// out = the parts' sum in their order, rounded once; 4 results a thread. The second output
// takes the results from `first` on.
template <bool H>
__global__ void __launch_bounds__(256)
join_kernel(const float* __restrict__ part, int split, int64_t n, uint16_t* __restrict__ out0, uint16_t* __restrict__ out1, int64_t first)
{
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    f32x4 v = *reinterpret_cast<const f32x4*>(part + i);
    for (int s = 1; s < split; ++s) v += *reinterpret_cast<const f32x4*>(part + s * n + i);
    uint16_t* o = i < first ? out0 + i : out1 + (i - first);
    *reinterpret_cast<u32x2*>(o) = u32x2{pack_x16<H>(v[0], v[1]), pack_x16<H>(v[2], v[3])};
}

// An empty sum over tokens: both weights' gradients are zero.
__global__ void __launch_bounds__(256)
zero_kernel(uint16_t* __restrict__ a, uint16_t* __restrict__ b, int64_t n)
{
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (i >= n) return;
    *reinterpret_cast<u32x4*>(a + i) = u32x4{0u, 0u, 0u, 0u};
    *reinterpret_cast<u32x4*>(b + i) = u32x4{0u, 0u, 0u, 0u};
}

template <int MODE, bool H>
hipError_t launch_tiles(const Geometry& g, const Tiling& t, const Args& a, hipStream_t st)
{
    TileArgs p = {a, g.T, g.D, g.F, g.act, t.na, t.nb, t.steps, t.per, t.split > 1 ? a.part : nullptr};
    const dim3 grid((unsigned)(cdiv(t.na * t.nb, 8) * 8), (unsigned)t.split);
    if (t.large) hipLaunchKernelGGL((tile_kernel<MODE, H, 2, 4, 8, 4>), grid, dim3(512), 0, st, p);
    else hipLaunchKernelGGL((tile_kernel<MODE, H, 2, 2, 4, 4>), grid, dim3(256), 0, st, p);
    return hipGetLastError();
}

template <bool H>
hipError_t join(const Tiling& t, const Args& a, int64_t n, uint16_t* out0, uint16_t* out1, int64_t first, hipStream_t st)
{
    if (t.split <= 1) return hipSuccess;
    hipLaunchKernelGGL(join_kernel<H>, dim3((unsigned)cdiv(n, 1024)), dim3(256), 0, st, a.part, t.split, n, out0, out1, first);
    return hipGetLastError();
}

template <bool H>
hipError_t backward(const Geometry& g, const BackwardPlan& p, const Args& a, hipStream_t st)
{
    hipError_t e = launch_tiles<kRecompute, H>(g, p.act, a, st);
    if (e != hipSuccess) return e;
    e = launch_tiles<kGradX, H>(g, p.dx, a, st);
    if (e != hipSuccess) return e;
    e = join<H>(p.dx, a, g.T * g.D, a.grad_x, a.grad_x, g.T * g.D, st);
    if (e != hipSuccess) return e;
    e = launch_tiles<kGradW, H>(g, p.dw, a, st);
    if (e != hipSuccess) return e;
    return join<H>(p.dw, a, 2 * (int64_t)g.F * g.D, a.grad_w_gate, a.grad_w_up, (int64_t)g.F * g.D, st);
}

}  // namespace

int launch_glu(const Geometry& g, const Args& a, void* stream)
{
    clear_pending_error();
    hipStream_t st = (hipStream_t)stream;
    return (int)(g.f16 ? launch_tiles<kForward, true>(g, forward_tiling(g), a, st)
                       : launch_tiles<kForward, false>(g, forward_tiling(g), a, st));
}

int launch_glu_backward(const Geometry& g, const BackwardPlan& p, const Args& a, void* stream)
{
    clear_pending_error();
    hipStream_t st = (hipStream_t)stream;
    if (g.T == 0) {
        const int64_t n = (int64_t)g.F * g.D;
        hipLaunchKernelGGL(zero_kernel, dim3((unsigned)cdiv(n, 2048)), dim3(256), 0, st, a.grad_w_gate, a.grad_w_up, n);
        return (int)hipGetLastError();
    }
    return (int)(g.f16 ? backward<true>(g, p, a, st) : backward<false>(g, p, a, st));
}

}  // namespace glu
}  // namespace mhc
