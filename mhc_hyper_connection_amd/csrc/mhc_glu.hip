// mhc_glu.hip -- gfx950 kernels of the gated projection and its backward.
//
//   forward   g = x Wg^T, u = x Wu^T, h = act(g) (.) u
//   backward  with dh = dL/dh: g and u again, dg = dh u act'(g), du = dh act(g), h = act(g) u,
//             dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x
// x [T, D], Wg and Wu [F, D], h and dh [T, F], bf16 or fp16 (template flag H); act(g) =
// g sigmoid(z) with z = g (SiLU, ACT 0) or 2 sqrt(2/pi) (g + 0.044715 g^3) (GELU's tanh form,
// ACT 1).
// Products accumulate in fp32 on the matrix cores; g, u and the activation stay in fp32
// registers; dg and du are rounded once to the 16-bit format, and so is each result. dg and du are
// operands of the next products: kept closer, as two 16-bit terms each, they would double
// the matrix work of all three gradients for a relative error of 1.7e-3 instead of 2.3e-3 (bf16). They
// have the format's range too: fp16 infinite from 65520 on, zero under 3e-8.
//
// Four products share one tiled kernel (tile_kernel): C = A B over a reduction of kBK = 64
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

struct TileArgs {
    Args t;
    int64_t T;
    int D, F, act;
    uint32_t na, nb;       // tiles along rows and columns
    uint32_t whole;        // tiles that one workgroup takes whole: the first of the tile order
    int64_t steps, per;    // stages in all, stages of a part of the other tiles
    uint32_t split;        // parts of each of those
    float* part;           // their fp32 results, [tile][part][block of results][thread]
};

// A wave's results of a gated tile, from f0 on and for tokens t0, t0 + 16, ..: lane values of g in
// acc[0 .. IA/2), of u in the rest, 8 consecutive f in a pair of blocks.
template <int MODE, bool H, int ACT, int IA, int IB>
__device__ __forceinline__ void gated_results(const TileArgs& p, int64_t f0, int64_t t0, const f32x4 (&acc)[IA][IB])
{
    const int64_t T = p.T;
    const int F = p.F;
    u32x4 dh[IB][IA / 4];
    if constexpr (MODE == kRecompute) {   // all of them on their way before the first is used
#pragma unroll
        for (int q = 0; q < IB; ++q)
#pragma unroll
            for (int i = 0; i < IA / 4; ++i) {
                const int64_t t = t0 + 16 * q < T ? t0 + 16 * q : T - 1, f = f0 + 32 * i < F ? f0 + 32 * i : 0;
                dh[q][i] = *reinterpret_cast<const u32x4*>(p.t.grad_h + t * F + f);
            }
    }
#pragma unroll
    for (int q = 0; q < IB; ++q) {
        const int64_t t = t0 + 16 * q;
#pragma unroll
        for (int i = 0; i < IA / 4; ++i) {
            const int64_t f = f0 + 32 * i;
            u32x4 hv, gv, uv;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float hh[2], dg[2], du[2];
#pragma unroll
                for (int l = 0; l < 2; ++l) {
                    const int r = 2 * e + l;                            // f + r
                    const float gg = acc[2 * i + r / 4][q][r % 4], uu = acc[IA / 2 + 2 * i + r / 4][q][r % 4];
                    const Act ac = activation<ACT>(gg);
                    hh[l] = ac.a * uu;
                    asm("" : "+v"(hh[l]));   // rounded to fp32 before fp16, in the forward as in the backward
                    if constexpr (MODE == kRecompute) {
                        const float d = l ? x16_hi<H>(dh[q][i][e]) : x16_lo<H>(dh[q][i][e]);
                        dg[l] = d * uu * ac.da;
                        du[l] = d * ac.a;
                    }
                }
                hv[e] = pack_x16<H>(hh[0], hh[1]);
                if constexpr (MODE == kRecompute) {
                    gv[e] = pack_x16<H>(dg[0], dg[1]);
                    uv[e] = pack_x16<H>(du[0], du[1]);
                }
            }
            if (t < T && f < F) {
                if (MODE == kForward || p.t.h) *reinterpret_cast<u32x4*>(p.t.h + t * F + f) = hv;
                if constexpr (MODE == kRecompute) {
                    *reinterpret_cast<u32x4*>(p.t.dgu + t * 2 * F + f) = gv;
                    *reinterpret_cast<u32x4*>(p.t.dgu + t * 2 * F + F + f) = uv;
                }
            }
        }
    }
}

// WA x WB waves of IA x IB 16 x 16 results each. A stage of the reduction is kBK = 64 positions,
// so that a direct load takes whole 128-byte lines of an operand contiguous along the
// reduction (with 32 the L2 saw twice the requests, and they bound the loop). LDS holds
// three stages of A and two of B. A wave's operands of half a stage (32 positions, the depth
// of one matrix-core instruction) are read while it multiplies the half before:
//   first half of stage m    read the second half of m, send off A's loads of stage m + 2
//   wait for the loads of stage m + 1, meet the other waves (whose reads of stage m are then done)
//   second half of stage m   read the first half of m + 1, send off B's loads of stage m + 2
// The reads and loads are dealt out between the products (loads sent off together held up
// every wave's next products: 6 % of the whole). Loads past the end of the reduction bring
// zeros.
template <int MODE, bool H, int WA, int WB, int IA, int IB>
__global__ void __launch_bounds__(64 * WA * WB, 2)
tile_kernel(TileArgs p)
{
    constexpr int NW = WA * WB;
    constexpr int AR = 16 * WA * IA, BC = 16 * WB * IB;          // rows and columns of the tile
    constexpr int ASZ = AR * 2 * kBK, BSZ = BC * 2 * kBK;        // bytes of a stage
    constexpr int QA = ASZ / 1024 / NW, QB = BSZ / 1024 / NW;    // direct loads of a wave per stage
    constexpr int RA = 3, RB = 2;                                // stages in LDS
    constexpr bool A_ACROSS = MODE == kGradX || MODE == kGradW;  // A contiguous across the reduction
    constexpr bool B_ACROSS = MODE == kGradW;
    constexpr bool GATED = MODE == kForward || MODE == kRecompute;
    static_assert(QA * 1024 * NW == ASZ && QB * 1024 * NW == BSZ, "whole direct loads");
    static_assert(!GATED || QA % 2 == 0, "a direct load is of one of the two weights");
    __shared__ __attribute__((aligned(1024))) char lds[RA * ASZ + RB * BSZ];

    Unit unit;
    if (!unit_of(blockIdx.x, p.na, p.nb, p.whole, p.split, &unit)) return;   // the padding of an XCD's run
    const int64_t ta = unit.a, tb = unit.b;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wa = wave / WB, wb = wave % WB;
    const int j = lane & 15, kg = lane >> 4;
    const int D = p.D, F = p.F;
    const int64_t T = p.T;
    const int half_steps = (F + kBK - 1) / kBK;                  // kGradX: stages of either weight
    // kGradW: the tiles of Wg's gradient, then those of Wu's
    const int64_t nbh = p.nb / 2;
    const int up = MODE == kGradW && tb >= nbh ? 1 : 0;
    const int64_t a0 = ta * (GATED ? AR / 2 : AR);               // first f (gated) or d
    const int64_t b0 = (tb - up * nbh) * BC;                     // first token, or f

    const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>(lds));
    const uint32_t ldsb = lds0 + RA * ASZ;

    // --- loads, 1 KiB each. Contiguous along the reduction: 8 LDS rows of 128 bytes; the 16-byte
    // chunk c of row r sits at c ^ s(r), s = (r / 2) % 8 for 16 rows in a run. The gated rows
    // are read 4 of every 8, and s = 2 ((r / 8) % 4) + (r / 2) % 2 numbers those the same way. The
    // LDS serves a 16-byte read in four turns of 16 lanes, the first of lanes 0-3, 12-15 and
    // 20-27, and each turn then meets all 64 banks once. Across: 64 / C rows of C chunks,
    // chunk c of position k at c ^ 2 ((k % 4) + 4 ((k / 8) % 2)). No conflicts are counted.
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
            const int r = 8 * i + lane / 8, c = (lane & 7) ^ (2 * ((r >> 3) & 3) + ((r >> 1) & 1));
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
            const int r = 8 * i + lane / 8, c = (lane & 7) ^ ((r >> 1) & 7);
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
    // load q of this wave's part of a stage of A, of B
    auto issue_a = [&](int64_t step, int slot, int q) __attribute__((always_inline)) {
        const uint32_t at = lds0 + slot * ASZ + (wave + q * NW) * 1024;
        if constexpr (GATED) {
            const int k = (int)(step * kBK);
            buffer_to_lds(q < QA / 2 ? dag : dau, k + ka[q] < D ? va[q] + 2 * k : kOutOfRange, at);
        } else if constexpr (MODE == kGradX) {
            const int hf = step >= half_steps ? 1 : 0;
            const int64_t k = (step - (int64_t)hf * half_steps) * kBK;
            buffer_to_lds(descriptor((hf ? p.t.w_up : p.t.w_gate) + k * D, rows_left(F, k) * (uint32_t)D * 2), va[q], at);
        } else {
            const uint32_t left = rows_left(T, step * kBK);
            buffer_to_lds(descriptor(p.t.x + (left ? step * kBK : 0) * D, left * (uint32_t)D * 2), va[q], at);
        }
    };
    auto issue_b = [&](int64_t step, int slot, int q) __attribute__((always_inline)) {
        const uint32_t at = ldsb + slot * BSZ + (wave + q * NW) * 1024;
        if constexpr (GATED) {
            const int k = (int)(step * kBK);
            buffer_to_lds(db, k + kb[q] < D ? vb[q] + 2 * k : kOutOfRange, at);
        } else if constexpr (MODE == kGradX) {
            const int hf = step >= half_steps ? 1 : 0;
            const int64_t k = (step - (int64_t)hf * half_steps) * kBK;
            buffer_to_lds(db, k + kb[q] < F ? vb[q] + (uint32_t)(2 * (k + (int64_t)hf * F)) : kOutOfRange, at);
        } else {
            const uint32_t left = rows_left(T, step * kBK);
            buffer_to_lds(descriptor(p.t.dgu + (left ? step * kBK : 0) * 2 * F, left * (uint32_t)F * 4), vb[q], at);
        }
    };

    // --- operand reads. Along: lane (j, kg) takes chunk kg of row j; the gated rows of a
    // pair of results (h = 0, 1) are 8 (j / 4) + 4 h + j % 4, so that a lane's two results
    // are 8 consecutive f.
    const uint32_t aoff = A_ACROSS ? (uint32_t)((8 * kg + (j >> 2)) * (AR * 2) +
                                                (((IA * 2 * wa + ((j & 3) >> 1)) ^ (2 * ((j >> 2) + 4 * (kg & 1)))) << 4) + (j & 1) * 8)
                                   : (uint32_t)((16 * wa * IA / 2 + 8 * (j >> 2) + (j & 3)) * 128 + ((kg ^ (j >> 1)) << 4));
    const uint32_t boff = B_ACROSS ? (uint32_t)((8 * kg + (j >> 2)) * (BC * 2) +
                                                (((IB * 2 * wb + ((j & 3) >> 1)) ^ (2 * ((j >> 2) + 4 * (kg & 1)))) << 4) + (j & 1) * 8)
                                   : (uint32_t)((16 * wb * IB + j) * 128 + ((kg ^ (j >> 1)) << 4));
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

    struct Operands {
        s16x8 a[IA], b[IB];
    };
    // the across reads' addresses, one instruction each, are formed anew for every half stage:
    // kept, all their sums with the slots would take more registers than there are
    uint32_t anow = aoff, bnow = boff;
    auto read_a = [&](int slot, int half, int i, Operands& o) __attribute__((always_inline)) {
        const uint32_t la = lds0 + slot * ASZ;
        if constexpr (A_ACROSS) o.a[i] = read_across((anow ^ (i << 5)) + (la + half * 32 * (AR * 2)), AR * 2);
        else {   // gated: results 0 .. IA/2 - 1 are the gate's, the rest the up projection's
            const int i2 = i % (IA / 2);
            o.a[i] = read_along(la + (aoff ^ (half << 6)) + (i < IA / 2 ? 0 : AR / 2 * 128) + (i2 / 2) * 4096 + (i2 % 2) * 512);
        }
    };
    auto read_b = [&](int slot, int half, int q, Operands& o) __attribute__((always_inline)) {
        const uint32_t lb = ldsb + slot * BSZ;
        if constexpr (B_ACROSS) o.b[q] = read_across((bnow ^ (q << 5)) + (lb + half * 32 * (BC * 2)), BC * 2);
        else o.b[q] = read_along(lb + (boff ^ (half << 6)) + q * 2048);
    };

    const int64_t m0 = unit.part < 0 ? 0 : unit.part * p.per;
    const int64_t m1 = unit.part < 0 || m0 + p.per > p.steps ? p.steps : m0 + p.per;
    Operands op[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int q = 0; q < QA; ++q) issue_a(m0 + s, s, q);
#pragma unroll
        for (int q = 0; q < QB; ++q) issue_b(m0 + s, s, q);
    }
    wait_loads_and_barrier<QA + QB>();
#pragma unroll
    for (int q = 0; q < IB; ++q) read_b(0, 0, q, op[0]);
#pragma unroll
    for (int i = 0; i < IA; ++i) read_a(0, 0, i, op[0]);
    // half of stage m (slot numbers s = m - m0): the products of `now` in IA parts, the reads of the next half
    // and the loads dealt out over them in order
    auto half = [&](int64_t m, int s, int h, const Operands& now, Operands& next) __attribute__((always_inline)) {
        constexpr int READS = IA + IB;
        const int rs = s + h;   // the stage whose half 1 - h is read
        if constexpr (A_ACROSS) asm volatile("" : "+v"(anow));
        if constexpr (B_ACROSS) asm volatile("" : "+v"(bnow));
#pragma unroll
        for (int i = 0; i < IA; ++i) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int r = i * READS / IA; r < (i + 1) * READS / IA; ++r) {
                if (r < IB) read_b(rs % RB, 1 - h, r, next);
                else read_a(rs % RA, 1 - h, r - IB, next);
            }
#pragma unroll
            for (int q = 0; q < IB; ++q) acc[i][q] = mfma<H>(now.a[i], now.b[q], acc[i][q]);
            __builtin_amdgcn_sched_barrier(0);
            if (h == 0) {
#pragma unroll
                for (int q = i * QA / IA; q < (i + 1) * QA / IA; ++q) issue_a(m + 2, (s + 2) % RA, q);
            } else {
#pragma unroll
                for (int q = i * QB / IA; q < (i + 1) * QB / IA; ++q) issue_b(m + 2, s % RB, q);
            }
        }
    };
    for (int64_t m = m0; m < m1; m += RA * RB) {
#pragma unroll
        for (int s = 0; s < RA * RB; ++s) {
            if (m + s < m1) {
                half(m + s, s, 0, op[0], op[1]);
                wait_loads_and_barrier<QA>();
                half(m + s, s, 1, op[1], op[0]);
            }
        }
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" : : : "memory");   // no load is left behind in LDS at the end

    // --- results: lane (j, kg) holds rows 4 kg .. 4 kg + 3 of column j of each 16 x 16 block
    if constexpr (GATED) {
        if (p.act) gated_results<MODE, H, 1, IA, IB>(p, a0 + 16 * wa * IA / 2 + 8 * kg, b0 + 16 * wb * IB + j, acc);
        else gated_results<MODE, H, 0, IA, IB>(p, a0 + 16 * wa * IA / 2 + 8 * kg, b0 + 16 * wb * IB + j, acc);
    } else if (unit.part < 0) {
        // through LDS, so that a wave stores whole rows of the tile ([column][row], rows
        // contiguous: grad_x [T][D], or a weight's gradient [F][D]): 2 AR bytes of a column and
        // 16 more, with which the 8-byte writes of 16 columns meet all banks
        constexpr int CS = 2 * AR + 16, OCT = AR / 8;
        static_assert(BC * CS <= RA * ASZ + RB * BSZ, "the tile fits in LDS");
        __syncthreads();   // every wave's last reads and loads are done (waited for above)
#pragma unroll
        for (int i = 0; i < IA; ++i)
#pragma unroll
            for (int q = 0; q < IB; ++q)
                *reinterpret_cast<u32x2*>(lds + (16 * (wb * IB + q) + j) * CS + (16 * (wa * IA + i) + 4 * kg) * 2) =
                    u32x2{pack_x16<H>(acc[i][q][0], acc[i][q][1]), pack_x16<H>(acc[i][q][2], acc[i][q][3])};
        __syncthreads();
        uint16_t* const out = MODE == kGradX ? p.t.grad_x : (up ? p.t.grad_w_up : p.t.grad_w_gate);
        const int o = tid % OCT;
        const int64_t d = a0 + 8 * o, ncol = MODE == kGradX ? T : F;
#pragma unroll
        for (int c = tid / OCT; c < BC; c += 64 * NW / OCT)
            if (d < D && b0 + c < ncol)
                *reinterpret_cast<u32x4*>(out + (b0 + c) * D + d) = *reinterpret_cast<const u32x4*>(lds + c * CS + 16 * o);
    } else {
        f32x4* const part = reinterpret_cast<f32x4*>(p.part) +
                            (int64_t)((unit.tile - p.whole) * p.split + unit.part) * (IA * IB * 64 * NW) + tid;
#pragma unroll
        for (int q = 0; q < IB; ++q) {
            if (b0 + 16 * (wb * IB + q) >= (MODE == kGradX ? T : (int64_t)F)) break;   // no such columns
#pragma unroll
            for (int i = 0; i < IA; ++i) part[(i * IB + q) * 64 * NW] = acc[i][q];
        }
    }
}

// The split tiles: a result is its parts' sum in their order, rounded once. Workgroup (tile,
// block): one 16 x 16 block of each of the tile's waves, laid out as tile_kernel left it;
// four parts on their way at a time.
template <int MODE, bool H, int WA, int WB, int IA, int IB>
__global__ void __launch_bounds__(64 * WA * WB)
join_kernel(TileArgs p)
{
    constexpr int NW = WA * WB, AR = 16 * WA * IA, BC = 16 * WB * IB, STRIDE = IA * IB * 64 * NW;
    Unit u;
    place(p.whole + blockIdx.x, p.na, p.nb, &u);
    const int i = blockIdx.y / IB, q = blockIdx.y % IB;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wa = wave / WB, wb = wave % WB;
    const uint32_t nbh = p.nb / 2;
    const int up = MODE == kGradW && u.b >= nbh ? 1 : 0;
    const int64_t d = (int64_t)u.a * AR + 16 * (wa * IA + i) + 4 * (lane >> 4);
    const int64_t c = (int64_t)(u.b - up * nbh) * BC + 16 * (wb * IB + q) + (lane & 15);
    if (c >= (MODE == kGradX ? p.T : (int64_t)p.F) || d >= p.D) return;
    const f32x4* part = reinterpret_cast<const f32x4*>(p.part) + (int64_t)blockIdx.x * p.split * STRIDE + blockIdx.y * (64 * NW) + tid;
    f32x4 v = part[0];
    uint32_t s = 1;
    for (; s + 4 <= p.split; s += 4) {
        f32x4 w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = part[(int64_t)(s + e) * STRIDE];
#pragma unroll
        for (int e = 0; e < 4; ++e) v += w[e];
    }
    for (; s < p.split; ++s) v += part[(int64_t)s * STRIDE];
    uint16_t* const out = MODE == kGradX ? p.t.grad_x : (up ? p.t.grad_w_up : p.t.grad_w_gate);
    *reinterpret_cast<u32x2*>(out + c * p.D + d) = u32x2{pack_x16<H>(v[0], v[1]), pack_x16<H>(v[2], v[3])};
}

// Few tokens (T <= 16 NT): reading the weights once is the whole cost. A workgroup takes 16 f of both
// projections and all tokens, its W waves every W-th run of 64 positions; their sums meet in
// LDS and are added in wave order. A wave keeps a ring of R stages of its own in LDS (32 weight
// rows and the tokens' rows, 128 bytes each, by direct loads of whole lines), so that it waits
// for its own loads only and meets the others once. (The same weights read straight into
// operand registers, 64 bytes of a row an instruction: 86 us against 70 at D = 7168, F = 14336,
// whatever the waves and loads in flight.) Rows past T or F and positions past D read as zeros.
template <int MODE, bool H, int NT, int W>
__global__ void __launch_bounds__(64 * W)
skinny_kernel(TileArgs p)
{
    constexpr int R = 3, ROWS = 32 + 16 * NT, STAGE = ROWS * 128, LOADS = ROWS / 8;
    static_assert(R * STAGE >= 2 * NT * 64 * 16, "a wave's sums fit where its stages were");
    __shared__ __attribute__((aligned(1024))) char lds[W * R * STAGE];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15, kg = lane >> 4, D = p.D, F = p.F;
    const int64_t f0 = (int64_t)blockIdx.x * 16;
    const uint32_t rows = (uint32_t)(F - f0 < 16 ? F - f0 : 16), line = (uint32_t)D * 2;
    const u32x4 dg_ = descriptor(p.t.w_gate + f0 * D, rows * line), du_ = descriptor(p.t.w_up + f0 * D, rows * line);
    const u32x4 dx_ = descriptor(p.t.x, (uint32_t)p.T * line);
    const uint32_t mine = __builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>(lds)) + wave * (R * STAGE);
    // load i of a stage: 8 rows; the 16-byte chunk c of row r sits at c ^ (r / 2) % 8, as in tile_kernel
    const int lr = lane / 8, lc = (lane & 7);
    auto issue = [&](int step, int slot) __attribute__((always_inline)) {
        const int k = step * 64;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int r = 8 * (i < 4 ? i % 2 : i - 4) + lr, c = lc ^ ((r >> 1) & 7);
            const uint32_t off = k + 8 * c < D ? (uint32_t)r * line + (uint32_t)(k + 8 * c) * 2 : kOutOfRange;
            buffer_to_lds(i < 2 ? dg_ : (i < 4 ? du_ : dx_), off, mine + slot * STAGE + i * 1024);
        }
    };
    const uint32_t at0 = mine + j * 128 + ((kg ^ (j >> 1)) << 4);
    f32x4 acc[2][NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[0][n] = acc[1][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int steps = (D + 63) / 64;
#pragma unroll
    for (int s = 0; s < R - 1; ++s) issue(wave + s * W, s);
    for (int k = wave; k < steps; k += R * W) {
#pragma unroll
        for (int s = 0; s < R; ++s) {
            if (k + s * W < steps) {
                issue(k + (s + R - 1) * W, (s + R - 1) % R);
                asm volatile("s_waitcnt vmcnt(%0)" : : "n"((R - 1) * LOADS) : "memory");
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t at = (at0 ^ (h << 6)) + s * STAGE;
                    const s16x8 g = *(const MHC_LDS s16x8*)(uintptr_t)at, u = *(const MHC_LDS s16x8*)(uintptr_t)(at + 2048);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const s16x8 x = *(const MHC_LDS s16x8*)(uintptr_t)(at + 4096 + n * 2048);
                        acc[0][n] = mfma<H>(g, x, acc[0][n]);
                        acc[1][n] = mfma<H>(u, x, acc[1][n]);
                    }
                }
                asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");   // read, before the slot is loaded again
            }
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
    // the sums, each wave's where its stages were
    auto red = [&](int w, int i) { return reinterpret_cast<f32x4*>(lds + w * (R * STAGE)) + i * 64; };
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        red(wave, 2 * n)[lane] = acc[0][n];
        red(wave, 2 * n + 1)[lane] = acc[1][n];
    }
    __syncthreads();
    if (wave >= NT) return;
    f32x4 g = red(0, 2 * wave)[lane], u = red(0, 2 * wave + 1)[lane];   // wave n: tokens 16 n ..
#pragma unroll
    for (int w = 1; w < W; ++w) {
        g += red(w, 2 * wave)[lane];
        u += red(w, 2 * wave + 1)[lane];
    }
    const int64_t t = 16 * wave + j, f = f0 + 4 * kg;
    if (t >= p.T || f >= F) return;
    u32x2 dh = {0u, 0u};
    if constexpr (MODE == kRecompute) dh = *reinterpret_cast<const u32x2*>(p.t.grad_h + t * F + f);
    float hh[4], dg[4], du[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const Act ac = p.act ? activation<1>(g[r]) : activation<0>(g[r]);
        hh[r] = ac.a * u[r];
        asm("" : "+v"(hh[r]));
        const float d = (r & 1) ? x16_hi<H>(dh[r >> 1]) : x16_lo<H>(dh[r >> 1]);
        dg[r] = d * u[r] * ac.da;
        du[r] = d * ac.a;
    }
    if (MODE == kForward || p.t.h)
        *reinterpret_cast<u32x2*>(p.t.h + t * F + f) = u32x2{pack_x16<H>(hh[0], hh[1]), pack_x16<H>(hh[2], hh[3])};
    if constexpr (MODE == kRecompute) {
        *reinterpret_cast<u32x2*>(p.t.dgu + t * 2 * F + f) = u32x2{pack_x16<H>(dg[0], dg[1]), pack_x16<H>(dg[2], dg[3])};
        *reinterpret_cast<u32x2*>(p.t.dgu + t * 2 * F + F + f) = u32x2{pack_x16<H>(du[0], du[1]), pack_x16<H>(du[2], du[3])};
    }
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

template <int MODE, bool H, int WA, int WB, int IA, int IB>
hipError_t launch_shape(const Geometry& g, const Tiling& t, const Args& a, hipStream_t st)
{
    const TileArgs p = {a, g.T, g.D, g.F, g.act, (uint32_t)t.na, (uint32_t)t.nb, (uint32_t)t.whole, t.steps, t.per, (uint32_t)t.split, a.part};
    hipLaunchKernelGGL((tile_kernel<MODE, H, WA, WB, IA, IB>), dim3((unsigned)t.blocks()), dim3(64 * WA * WB), 0, st, p);
    hipError_t e = hipGetLastError();
    if constexpr (MODE == kGradX || MODE == kGradW) {
        if (e == hipSuccess && t.rest() > 0) {
            hipLaunchKernelGGL((join_kernel<MODE, H, WA, WB, IA, IB>), dim3((unsigned)t.rest(), IA * IB), dim3(64 * WA * WB), 0, st, p);
            e = hipGetLastError();
        }
    }
    return e;
}

template <int MODE, bool H>
hipError_t launch_tiles(const Geometry& g, const Tiling& t, const Args& a, hipStream_t st)
{
    if constexpr (MODE == kForward || MODE == kRecompute) {
        if (g.skinny()) {
            const TileArgs p = {a, g.T, g.D, g.F, g.act};
            const dim3 grid((unsigned)cdiv(g.F, 16)), block(256);
            if (g.T <= 16) hipLaunchKernelGGL((skinny_kernel<MODE, H, 1, 4>), grid, block, 0, st, p);
            else if (g.T <= 32) hipLaunchKernelGGL((skinny_kernel<MODE, H, 2, 4>), grid, block, 0, st, p);
            else hipLaunchKernelGGL((skinny_kernel<MODE, H, 4, 4>), grid, block, 0, st, p);
            return hipGetLastError();
        }
    }
    return t.large ? launch_shape<MODE, H, 2, 4, 8, 4>(g, t, a, st) : launch_shape<MODE, H, 2, 2, 4, 4>(g, t, a, st);
}

template <bool H>
hipError_t backward(const Geometry& g, const BackwardPlan& p, const Args& a, hipStream_t st)
{
    hipError_t e = launch_tiles<kRecompute, H>(g, p.act, a, st);
    if (e == hipSuccess) e = launch_tiles<kGradX, H>(g, p.dx, a, st);
    if (e == hipSuccess) e = launch_tiles<kGradW, H>(g, p.dw, a, st);
    return e;
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
