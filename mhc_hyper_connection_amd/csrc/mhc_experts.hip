// mhc_experts.hip -- gfx950 kernels of the products with 4-bit weights.
//
//   product       y = x w^T
//   experts_glu   h[p] = act(x[p / k] Wg[e]^T) (.) (x[p / k] Wu[e]^T)   for the pairs p of each expert e
//   experts_down  y[t] = sum_j weights[t, j] (h[t, j] Wd[e]^T)
// x, h and the weights are microscaled 4-bit floats (mhc_mxfp4_device.h); the matrix instruction takes
// codes and scale bytes as they are in memory: a lane's 16 bytes of codes are one block of 32
// values, and its scale byte that block's. Products accumulate in fp32; the activation and the
// weighted sum are fp32, one rounding to the 16-bit result.
//
// A unit of work is a run of weight rows and up to a tile's columns of one expert's pairs, which are
// gathered by the plan's list as their x rows are loaded. Pairs without an expert are a bucket of their own
// behind the last expert's: their results are zeros.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "mhc_experts_plan.h"
#include "mhc_tile_device.h"

namespace mhc {
namespace experts {
namespace {

enum Out { kOutBf16, kOutF16, kOutF32 };

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

constexpr int kLine = 128;            // bytes of a row's codes in a stage: 256 values, 8 scale bytes

// BA, BB: the bytes of sa and sb that hold the scales
template <int BA, int BB>
__device__ __forceinline__ f32x4 mfma4(i32x4 a, i32x4 b, f32x4 c, int sa, int sb)
{
    const i32x4 z = {0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_shufflevector(a, z, 0, 1, 2, 3, 4, 5, 6, 7),
                                                            __builtin_shufflevector(b, z, 0, 1, 2, 3, 4, 5, 6, 7),
                                                            c, 4, 4, BA, sa, BB, sb);
}
// 64 lanes x 4 bytes from the buffer to LDS at `lds` (lane l to lds + 4 l); as buffer_to_lds.
__device__ __forceinline__ void word_to_lds(u32x4 desc, uint32_t offset, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds" : : "v"(offset), "s"(desc), "s"(lds) : "memory");
}

template <int N>
struct Number {
    static constexpr int value = N;
};

struct TileArgs {
    Args t;
    int64_t P;
    int E, R, act;
    uint32_t kb, sb;       // bytes of a row's codes and scales
    uint32_t na, share;
    uint32_t x_rows;
};

// The unit of this workgroup: of expert e the units' row a and the pairs [first, first + cols). An
// XCD (workgroups b, b + 8, ..) takes a contiguous run of the units. The experts' buckets are counted from the plan's
// offsets, which are bounded here: whatever they hold, pairs stay in [0, P).
struct Unit {
    int e;
    uint32_t a;
    int64_t first;
    int cols;
};
template <int BC>
__device__ __forceinline__ bool find_unit(const TileArgs& p, Unit* u)
{
    const int lane = threadIdx.x & 63;
    const uint32_t xcd = blockIdx.x % 8, i = blockIdx.x / 8;
    auto bucket = [&](int e, int64_t* begin, int64_t* end) {
        const int64_t b = e <= p.E ? p.t.offsets[e] : p.P, n = e < p.E ? p.t.offsets[e + 1] : p.P;
        *begin = b < 0 ? 0 : (b > p.P ? p.P : b);
        *end = n < *begin ? *begin : (n > p.P ? p.P : n);
        return (int)((*end - *begin + BC - 1) / BC);
    };
    int64_t begin, end;
    uint32_t total = 0, nb, at;
    if (!p.t.offsets) {
        total = (uint32_t)((p.P + BC - 1) / BC);
    } else {
        for (int e0 = 0; e0 <= p.E; e0 += 64) {
            int n = bucket(e0 + lane, &begin, &end);
#pragma unroll
            for (int d = 1; d < 64; d *= 2) n += __shfl_xor(n, d);
            total += (uint32_t)__builtin_amdgcn_readfirstlane(n);
        }
    }
    const uint32_t units = total * p.na, per = (units + 7) / 8, unit = xcd * per + i;
    if (i >= per || unit >= units) return false;
    uint32_t b;
    if (!p.t.offsets) {
        place(unit, p.na, total, &u->a, &b);
        u->e = 0;
        u->first = (int64_t)b * BC;
        u->cols = (int)(p.P - u->first < BC ? p.P - u->first : BC);
        return true;
    }
    const uint32_t q = unit / p.na;
    at = 0;
    for (int e0 = 0; e0 <= p.E; e0 += 64) {
        const int n = bucket(e0 + lane, &begin, &end);
        int scan = n;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(scan, d);
            if (lane >= d) scan += o;
        }
        const uint64_t past = __ballot(q < at + (uint32_t)scan);
        if (past) {
            const int l = __builtin_ctzll(past);
            nb = (uint32_t)__builtin_amdgcn_readlane(n, l);
            at += (uint32_t)(__builtin_amdgcn_readlane(scan, l) - (int)nb);
            const int b0 = __builtin_amdgcn_readlane((int)begin, l), b1 = __builtin_amdgcn_readlane((int)end, l);
            place(unit - at * p.na, p.na, nb, &u->a, &b);
            u->e = e0 + l;
            u->first = b0 + (int64_t)b * BC;
            u->cols = (int)(b1 - u->first < BC ? b1 - u->first : BC);
            return true;
        }
        at += (uint32_t)__builtin_amdgcn_readlane(scan, 63);
    }
    return false;
}
template <int BC>
__device__ __forceinline__ bool unit_of(const TileArgs& p, Unit* u)
{
    Unit v = {0, 0, 0, 0};
    if (!find_unit<BC>(p, &v)) return false;
    // the same in every lane: to scalar registers, which the direct loads' descriptors have to be in
    auto scalar = [](int x) {
        int s;
        asm volatile("s_nop 1\n\tv_readfirstlane_b32 %0, %1" : "=s"(s) : "v"(x));
        return s;
    };
    u->e = scalar(v.e);
    u->a = (uint32_t)scalar((int)v.a);
    u->first = (int64_t)(uint32_t)scalar((int)v.first);    // under 2^31
    u->cols = scalar(v.cols);
    return true;
}
// The pair in column c of the unit; -1 past its columns (and for what is no pair).
__device__ __forceinline__ int64_t pair_of(const TileArgs& p, const Unit& u, int c)
{
    if (c >= u.cols) return -1;
    const int64_t i = u.first + c;
    if (!p.t.pairs) return i;
    const int64_t q = p.t.pairs[i];
    return q < 0 || q >= p.P ? -1 : q;
}

// Eight results of consecutive weight rows from r on, or four of them, of a pair.
template <int OUT, int N>
__device__ __forceinline__ void store_results(const TileArgs& p, int64_t pair, int64_t r, const float (&v)[N])
{
    if constexpr (OUT == kOutF32) {
#pragma unroll
        for (int h = 0; h < N / 4; ++h)
            *reinterpret_cast<f32x4*>(p.t.part + pair * p.R + r + 4 * h) = f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
    } else {
        uint16_t* const out = static_cast<uint16_t*>(p.t.out) + pair * p.R + r;
        uint32_t w[N / 2];
#pragma unroll
        for (int e = 0; e < N / 2; ++e) w[e] = pack_x16<OUT == kOutF16>(v[2 * e], v[2 * e + 1]);
        if constexpr (N == 8) *reinterpret_cast<u32x4*>(out) = u32x4{w[0], w[1], w[2], w[3]};
        else *reinterpret_cast<u32x2*>(out) = u32x2{w[0], w[1]};
    }
}

// WA x WB waves of IA x IB 16 x 16 results each; rows: weights (gated: gate and up side by side, so that a wave
// holds both of the same f), columns: pairs. A stage of the reduction is 256 values: a row's 128 bytes
// of codes, which direct loads take as whole lines. LDS holds two stages of them, and the scales of two groups of
// four stages: 32 bytes of a row at a time, since a row's piece of scales takes a request of its own however short it
// is (8 bytes at a time, the requests were as many as those of the codes: 860 us instead of 720 at 65536 pairs, D = 4096,
// F = 2048). A wave's operands of half a stage (128 values, the depth of one matrix instruction) are read while it
// multiplies the half before:
//   first half of stage m    read the second half of m
//   wait for all loads, meet the other waves (whose reads of stage m are then done)
//   second half of stage m   read the first half of m + 1, send off the loads of stage m + 2 and (but for the
//                            group's last stage) a third of those of the next group's scales
// Loads past the end of the reduction bring zeros.
template <bool GATED, int OUT, int WA, int WB, int IA, int IB>
__global__ void __launch_bounds__(64 * WA * WB, WA * WB == 4 && IA * IB == 64 ? 1 : 2)
tile_kernel(TileArgs p)
{
    constexpr int NW = WA * WB;
    constexpr int AR = 16 * WA * IA, BC = 16 * WB * IB;
    constexpr int ASZ = AR * kLine, BSZ = BC * kLine, STAGE = ASZ + BSZ, GROUP = (AR + BC) * 32;
    constexpr int QA = ASZ / 1024 / NW, QB = BSZ / 1024 / NW, SA = AR / 8 / NW, SB = BC / 8 / NW;   // a wave's loads; of a group's scales
    static_assert(QA * 1024 * NW == ASZ && QB * 1024 * NW == BSZ && SA * 8 * NW == AR && SB * 8 * NW == BC, "whole direct loads");
    static_assert(!GATED || (QA % 2 == 0 && SA % 2 == 0), "a direct load is of one of the two weights");
    static_assert(IA % (GATED ? 4 : 2) == 0, "blocks in pairs");
    __shared__ __attribute__((aligned(1024))) char lds[2 * STAGE + 2 * GROUP];

    Unit u;
    if (!unit_of<BC>(p, &u)) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wa = wave / WB, wb = wave % WB;
    const int j = lane & 15, kg = lane >> 4;
    const uint32_t kb = p.kb, sb = p.sb;
    constexpr int ROWS = GATED ? AR / 2 : AR;                    // of one weight
    const int64_t a0 = (int64_t)u.a * ROWS, R = p.R;
    const uint32_t arow = (uint32_t)(R - a0 < ROWS ? R - a0 : ROWS);
    const bool routed = u.e < p.E;

    f32x4 acc[IA][IB];
#pragma unroll
    for (int i = 0; i < IA; ++i)
#pragma unroll
        for (int q = 0; q < IB; ++q) acc[i][q] = f32x4{0.f, 0.f, 0.f, 0.f};

    if (routed) {
        const int64_t w0 = u.e * R + a0;
        const u32x4 dc0 = descriptor(p.t.w_codes[0] + w0 * kb, arow * kb);
        const u32x4 dc1 = GATED ? descriptor(p.t.w_codes[1] + w0 * kb, arow * kb) : dc0;
        const u32x4 ds0 = descriptor(p.t.w_scales[0] + w0 * sb, arow * sb);
        const u32x4 ds1 = GATED ? descriptor(p.t.w_scales[1] + w0 * sb, arow * sb) : ds0;
        const u32x4 dxc = descriptor(p.t.x_codes, p.x_rows * kb), dxs = descriptor(p.t.x_scales, p.x_rows * sb);
        const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>(lds));

        // --- loads of codes, 1 KiB each: 8 LDS rows of 128 bytes. A lane group kg takes the blocks 2 kg and 2 kg + 1 of a
        // stage, one in each half, so that their scales are neighbours; the 16-byte chunk c of row r sits at c ^ s(r), where with
        // the reading lane's number j of 16, s has the bits (j >> 3 ^ j >> 2, j >> 1, j >> 2): each of the four turns of a 16-byte
        // read (the first of lanes 0-3, 12-15 and 20-27) then meets all banks once.
        auto swizzle = [](int j) __attribute__((always_inline)) { return (((j >> 3) ^ (j >> 2)) & 1) * 4 + (j & 2) + ((j >> 2) & 1); };
        auto x_row = [=](int c) __attribute__((always_inline)) {
            const int64_t q = pair_of(p, u, c);
            return q < 0 ? -1 : (int)((uint32_t)q / p.share);
        };
        // the weight rows of a pair of results are 8 (j / 4) + 4 h + j % 4
        const int r0 = 8 * wave + lane / 8;                      // this lane's row of a wave's first load; the others' have the same swizzle
        const uint32_t ka = 16 * ((lane & 7) ^ swizzle(((r0 >> 1) & 12) + (r0 & 3))), kx = 16 * ((lane & 7) ^ swizzle(r0 & 15));
        static_assert(NW % 4 == 0, "rows 32 apart");
        uint32_t va[QA], vb[QB], vs[SB];
#pragma unroll
        for (int q = 0; q < QA; ++q) va[q] = (uint32_t)((r0 + 8 * NW * q) % ROWS) * kb + ka;
#pragma unroll
        for (int q = 0; q < QB; ++q) {
            const int x = x_row(r0 + 8 * NW * q);
            vb[q] = x < 0 ? kOutOfRange : (uint32_t)x * kb + kx;
            if (q < SB) vs[q] = x < 0 ? kOutOfRange : (uint32_t)x * sb;
        }
        static_assert(SB == QB && SA == QA, "a load of scales has the rows of one of codes");
        // scales, 8 rows of 8 words a load; the pair of words of a row's stage n of 4 sits at n ^ (r / 8) % 4, so that the
        // rows of a block of results, 8 apart or 16 in a run, meet different banks
        const uint32_t ks = 4 * ((lane & 7) ^ (2 * (wave & 3)));
        // load q of this wave's part of a stage of the weights, of the pairs, of either's scales
        auto issue_a = [=](int step, int slot, int q) __attribute__((always_inline)) {
            const uint32_t k = (uint32_t)step * kLine;
            buffer_to_lds(!GATED || q < QA / 2 ? dc0 : dc1, k + ka < kb ? va[q] + k : kOutOfRange, lds0 + slot * STAGE + (wave + q * NW) * 1024);
        };
        auto issue_b = [=](int step, int slot, int q) __attribute__((always_inline)) {
            const uint32_t k = (uint32_t)step * kLine;
            buffer_to_lds(dxc, k + kx < kb ? vb[q] + k : kOutOfRange, lds0 + slot * STAGE + ASZ + (wave + q * NW) * 1024);
        };
        auto issue_s = [=](int group, uint32_t slot, int n) __attribute__((always_inline)) {
            const uint32_t s = (uint32_t)group * 32 + ks, at = lds0 + 2 * STAGE + slot;
            if (n < SA) word_to_lds(!GATED || n < SA / 2 ? ds0 : ds1, s < sb ? (uint32_t)((r0 + 8 * NW * n) % ROWS) * sb + s : kOutOfRange, at + (wave + NW * n) * 256);
            else word_to_lds(dxs, s < sb ? vs[n - SA] + s : kOutOfRange, at + (wave + NW * n) * 256);
        };

        // --- operand reads: lane (j, kg) takes block 2 kg + half of row j of each block of 16
        constexpr int WR = GATED ? 16 * IA / 2 : 16 * IA;       // a wave's rows of one weight
        const uint32_t arow0 = (uint32_t)(wa * WR + 8 * (j >> 2) + (j & 3)), brow0 = (uint32_t)(16 * wb * IB + j);
        const uint32_t chunk = (uint32_t)((2 * kg) ^ swizzle(j)) << 4;
        const uint32_t aoff = arow0 * kLine + chunk, boff = ASZ + brow0 * kLine + chunk;
        const uint32_t asc = lds0 + 2 * STAGE + arow0 * 32 + (j >> 2) * 8 + 2 * kg, bsc = lds0 + 2 * STAGE + (AR + brow0) * 32 + (j >> 3) * 8 + 2 * kg;
        struct Operands {
            i32x4 a[IA], b[IB];
        };
        struct Scales {                // of a stage: two bytes, one for each half, of two blocks of results in a word
            u16x2 a[IA / 2], b[IB / 2];
        };
        auto row_of = [](int i) __attribute__((always_inline)) {
            const int i2 = GATED ? i % (IA / 2) : i;
            return (GATED && i >= IA / 2 ? ROWS : 0) + (i2 / 2) * 32 + (i2 % 2) * 4;
        };
        auto read_a = [=](int slot, int half, int i, Operands& o) __attribute__((always_inline)) {
            o.a[i] = *(const MHC_LDS i32x4*)(uintptr_t)(lds0 + slot * STAGE + (aoff ^ (half << 4)) + row_of(i) * kLine);
        };
        auto read_b = [=](int slot, int half, int q, Operands& o) __attribute__((always_inline)) {
            o.b[q] = *(const MHC_LDS i32x4*)(uintptr_t)(lds0 + slot * STAGE + (boff ^ (half << 4)) + q * 16 * kLine);
        };
        // of stage n of the group in `slot`
        auto read_sa = [=](uint32_t slot, int n, int i, Scales& o) __attribute__((always_inline)) {
            o.a[i / 2][i % 2] = *(const MHC_LDS uint16_t*)(uintptr_t)((asc ^ (n << 3)) + slot + row_of(i) * 32);
        };
        auto read_sb = [=](uint32_t slot, int n, int q, Scales& o) __attribute__((always_inline)) {
            o.b[q / 2][q % 2] = *(const MHC_LDS uint16_t*)(uintptr_t)((bsc ^ ((n ^ 2 * (q & 1)) << 3)) + slot + q * 16 * 32);
        };

        const int steps = (int)((kb + kLine - 1) / kLine);
        Operands op[2];
        Scales sc[2];
#pragma unroll
        for (int n = 0; n < SA + SB; ++n) issue_s(0, 0, n);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int q = 0; q < QA; ++q) issue_a(s, s, q);
#pragma unroll
            for (int q = 0; q < QB; ++q) issue_b(s, s, q);
        }
        wait_loads_and_barrier<QA + QB>();
#pragma unroll
        for (int q = 0; q < IB; ++q) read_b(0, 0, q, op[0]), read_sb(0, 0, q, sc[0]);
#pragma unroll
        for (int i = 0; i < IA; ++i) read_a(0, 0, i, op[0]), read_sa(0, 0, i, sc[0]);
        // half H2 of stage m = 4 group + n: the products of `now` in IA parts, the reads of the next half (and of the next
        // stage's scales) and the loads dealt out over them; `slot`: where the next stage's scales are, `other`: the next group's
        auto half = [&](auto number, int m, int n, const Operands& now, Operands& next, const Scales& sn, Scales& sx, uint32_t slot,
                        uint32_t other) __attribute__((always_inline)) {
            constexpr int READS = IA + IB, H2 = decltype(number)::value;
            const int s = n % 2, rs = (s + H2) % 2;
            // the next group's scales go with the first three stages: they have to be there when the fourth reads them
            const int QN = n < 3 ? (n + 1) * (SA + SB) / 3 - n * (SA + SB) / 3 : 0;
#pragma unroll
            for (int i = 0; i < IA; ++i) {
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int r = i * READS / IA; r < (i + 1) * READS / IA; ++r) {
                    if (r < IB) {
                        read_b(rs, 1 - H2, r, next);
                        if (H2) read_sb(slot, (n + 1) % 4, r, sx);
                    } else {
                        read_a(rs, 1 - H2, r - IB, next);
                        if (H2) read_sa(slot, (n + 1) % 4, r - IB, sx);
                    }
                }
                const int sa = __builtin_bit_cast(int, sn.a[i / 2]);
#pragma unroll
                for (int q = 0; q < IB; ++q) {
                    const int sb2 = __builtin_bit_cast(int, sn.b[q / 2]);
                    f32x4& c = acc[i][q];
                    if (i % 2 == 0) c = q % 2 == 0 ? mfma4<H2, H2>(now.a[i], now.b[q], c, sa, sb2) : mfma4<H2, 2 + H2>(now.a[i], now.b[q], c, sa, sb2);
                    else c = q % 2 == 0 ? mfma4<2 + H2, H2>(now.a[i], now.b[q], c, sa, sb2) : mfma4<2 + H2, 2 + H2>(now.a[i], now.b[q], c, sa, sb2);
                }
                __builtin_amdgcn_sched_barrier(0);
                if (H2 == 1) {
#pragma unroll
                    for (int q = i * QA / IA; q < (i + 1) * QA / IA; ++q) issue_a(m + 2, s, q);
#pragma unroll
                    for (int q = i * QB / IA; q < (i + 1) * QB / IA; ++q) issue_b(m + 2, s, q);
#pragma unroll
                    for (int q = i * QN / IA; q < (i + 1) * QN / IA; ++q) issue_s(m / 4 + 1, other, n * (SA + SB) / 3 + q);
                }
            }
        };
        uint32_t slot = 0;
        for (int m = 0; m < steps; m += 4) {
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                if (m + n < steps) {
                    half(Number<0>{}, m + n, n, op[0], op[1], sc[n % 2], sc[1 - n % 2], slot, slot ^ GROUP);
                    wait_loads_and_barrier<0>();
                    half(Number<1>{}, m + n, n, op[1], op[0], sc[n % 2], sc[1 - n % 2], n == 3 ? slot ^ GROUP : slot, slot ^ GROUP);
                }
            }
            slot ^= GROUP;
        }
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" : : : "memory");   // no load is left behind in LDS at the end
    }

    // --- results: lane (j, kg) holds rows 4 kg .. 4 kg + 3 of column j of each 16 x 16 block
#pragma unroll
    for (int q = 0; q < IB; ++q) {
        const int64_t pair = pair_of(p, u, 16 * (wb * IB + q) + j);
        if (pair < 0) continue;
        if constexpr (GATED) {
#pragma unroll
            for (int i = 0; i < IA / 4; ++i) {
                const int64_t f = a0 + wa * (16 * IA / 2) + 32 * i + 8 * kg;
                float v[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const float g = acc[2 * i + r / 4][q][r % 4], up = acc[IA / 2 + 2 * i + r / 4][q][r % 4];
                    v[r] = (p.act ? activation<1>(g) : activation<0>(g)).a * up;
                }
                if (f < R) store_results<OUT>(p, pair, f, v);
            }
        } else {
#pragma unroll
            for (int i = 0; i < IA / 2; ++i) {
                const int64_t f = a0 + wa * (16 * IA) + 32 * i + 8 * kg;
                float v[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) v[r] = acc[2 * i + r / 4][q][r % 4];
                if (f < R) store_results<OUT>(p, pair, f, v);
            }
        }
    }
}

// Few pairs of an expert (16 NT at most to a unit): reading the weights once is the whole cost. A
// workgroup takes 32 weight rows (gated: 16 of either weight), its W waves every W-th stage of 256 values; their
// sums meet in LDS and are added in wave order. A wave keeps a ring of three stages of its own in LDS,
// so that it waits for its own loads only and meets the others once.
template <bool GATED, int OUT, int NT>
__global__ void __launch_bounds__(256)
skinny_kernel(TileArgs p)
{
    constexpr int W = 4, RING = 3, ROWS = 32 + 16 * NT;
    // loads of scales: 16 rows of a gated pair of weights each (half a load, the other lanes idle) or 32 rows;
    // the pairs' 16 or 32 rows each
    constexpr int SW = GATED ? 2 : 1, SX = (NT + 1) / 2, SXB = NT == 1 ? 128 : 256;
    constexpr int CODES = ROWS * kLine, STAGE = CODES + 256 + SX * SXB, LOADS = ROWS / 8 + SW + SX;
    static_assert(RING * STAGE >= 2 * NT * 64 * 16, "a wave's sums fit where its stages were");
    __shared__ __attribute__((aligned(1024))) char lds[W * RING * STAGE];
    Unit u;
    if (!unit_of<16 * NT>(p, &u)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15, kg = lane >> 4;
    const uint32_t kb = p.kb, sb = p.sb;
    constexpr int WR = GATED ? 16 : 32;                          // rows of one weight
    const int64_t a0 = (int64_t)u.a * WR, R = p.R;
    const uint32_t arow = (uint32_t)(R - a0 < WR ? R - a0 : WR);

    f32x4 acc[2][NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[0][n] = acc[1][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (u.e < p.E) {
        const int64_t w0 = u.e * R + a0;
        const u32x4 dc0 = descriptor(p.t.w_codes[0] + w0 * kb, arow * kb), ds0 = descriptor(p.t.w_scales[0] + w0 * sb, arow * sb);
        const u32x4 dc1 = GATED ? descriptor(p.t.w_codes[1] + w0 * kb, arow * kb) : dc0;
        const u32x4 ds1 = GATED ? descriptor(p.t.w_scales[1] + w0 * sb, arow * sb) : ds0;
        const u32x4 dxc = descriptor(p.t.x_codes, p.x_rows * kb), dxs = descriptor(p.t.x_scales, p.x_rows * sb);
        const uint32_t mine = __builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>(lds)) + wave * (RING * STAGE);
        // a load of codes takes 8 rows; chunk c of row r sits at c ^ (r / 2) % 8
        const int lr = lane / 8, lc = lane & 7;
        uint32_t vx[2 * NT], kx[2 * NT], vs[SX], ks[SX];
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) {
            const int r = 8 * i + lr, c = lc ^ ((r >> 1) & 7);
            const int64_t q = pair_of(p, u, r);
            kx[i] = q < 0 ? kb : 16 * c;                         // no such column: past the end at once
            vx[i] = q < 0 ? 0u : ((uint32_t)q / p.share) * kb + kx[i];
        }
#pragma unroll
        for (int i = 0; i < SX; ++i) {
            const int r = 32 * i + lane / 2;
            const int64_t q = r < 16 * NT ? pair_of(p, u, r) : -1;
            ks[i] = q < 0 ? sb : 4 * (lane & 1);
            vs[i] = q < 0 ? 0u : ((uint32_t)q / p.share) * sb + ks[i];
        }
        auto issue = [=](int step, int slot) __attribute__((always_inline)) {
            const uint32_t k = (uint32_t)step * kLine, s = (uint32_t)step * 8, at = mine + slot * STAGE;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 8 * (GATED ? i % 2 : i) + lr, c = lc ^ ((r >> 1) & 7);
                buffer_to_lds(GATED && i >= 2 ? dc1 : dc0, k + 16 * c < kb ? (uint32_t)r * kb + k + 16 * c : kOutOfRange, at + i * 1024);
            }
#pragma unroll
            for (int i = 0; i < 2 * NT; ++i)
                buffer_to_lds(dxc, k + kx[i] < kb ? vx[i] + k : kOutOfRange, at + (4 + i) * 1024);
            const uint32_t w = s + 4 * (lane & 1);               // rows past the weight's are out of range
#pragma unroll
            for (int i = 0; i < SW; ++i)
                if (!GATED || lane < 32)
                    word_to_lds(i ? ds1 : ds0, w < sb ? (uint32_t)(lane / 2) * sb + w : kOutOfRange, at + CODES + i * 128);
#pragma unroll
            for (int i = 0; i < SX; ++i)
                if (NT > 1 || lane < 32)
                    word_to_lds(dxs, s + ks[i] < sb ? vs[i] + s : kOutOfRange, at + CODES + 256 + i * SXB);
        };
        const uint32_t at0 = mine + j * kLine + ((kg ^ (j >> 1)) << 4), sc0 = mine + CODES + j * 8 + kg;
        const int steps = (int)((kb + kLine - 1) / kLine);
#pragma unroll
        for (int s = 0; s < RING - 1; ++s) issue(wave + s * W, s);
        for (int k = wave; k < steps; k += RING * W) {
#pragma unroll
            for (int s = 0; s < RING; ++s) {
                if (k + s * W < steps) {
                    issue(k + (s + RING - 1) * W, (s + RING - 1) % RING);
                    asm volatile("s_waitcnt vmcnt(%0)" : : "n"((RING - 1) * LOADS) : "memory");
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t at = (at0 ^ (h << 6)) + s * STAGE, sc = sc0 + s * STAGE + 4 * h;
                        const i32x4 w0v = *(const MHC_LDS i32x4*)(uintptr_t)at, w1v = *(const MHC_LDS i32x4*)(uintptr_t)(at + 16 * kLine);
                        const int s0 = *(const MHC_LDS uint8_t*)(uintptr_t)sc, s1 = *(const MHC_LDS uint8_t*)(uintptr_t)(sc + 128);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const i32x4 x = *(const MHC_LDS i32x4*)(uintptr_t)(at + (32 + 16 * n) * kLine);
                            const int sx = *(const MHC_LDS uint8_t*)(uintptr_t)(sc + 256 + n * 128);
                            acc[0][n] = mfma4<0, 0>(w0v, x, acc[0][n], s0, sx);
                            acc[1][n] = mfma4<0, 0>(w1v, x, acc[1][n], s1, sx);
                        }
                    }
                    asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");   // read, before the slot is loaded again
                }
            }
        }
        asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
    }
    // the sums, each wave's where its stages were
    auto red = [&](int w, int i) { return reinterpret_cast<f32x4*>(lds + w * (RING * STAGE)) + i * 64; };
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        red(wave, 2 * n)[lane] = acc[0][n];
        red(wave, 2 * n + 1)[lane] = acc[1][n];
    }
    __syncthreads();
    if (wave >= NT) return;
    f32x4 v0 = red(0, 2 * wave)[lane], v1 = red(0, 2 * wave + 1)[lane];   // wave n: columns 16 n ..
#pragma unroll
    for (int w = 1; w < W; ++w) {
        v0 += red(w, 2 * wave)[lane];
        v1 += red(w, 2 * wave + 1)[lane];
    }
    const int64_t pair = pair_of(p, u, 16 * wave + j), r = a0 + 4 * kg;
    if (pair < 0) return;
    if constexpr (GATED) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (p.act ? activation<1>(v0[e]) : activation<0>(v0[e])).a * v1[e];
        if (r < R) store_results<OUT>(p, pair, r, v);
    } else {
        const float lo[4] = {v0[0], v0[1], v0[2], v0[3]}, hi[4] = {v1[0], v1[1], v1[2], v1[3]};
        if (r < R) store_results<OUT>(p, pair, r, lo);
        if (r + 16 < R) store_results<OUT>(p, pair, r + 16, hi);
    }
}

// A token's results by its weights: fp32 terms in the order of its slots, one rounding. A thread takes eight values.
template <bool H>
__global__ void __launch_bounds__(256)
combine_kernel(const float* __restrict__ part, const float* __restrict__ weights, uint16_t* __restrict__ out, int64_t T, int k, int R)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int octets = R / 8;
    const int64_t t = i / octets;
    if (t >= T) return;
    const int64_t r = (i - t * octets) * 8;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = 0; s < k; ++s) {
        const f32x4* const row = reinterpret_cast<const f32x4*>(part + (t * k + s) * R + r);
        const f32x4 a = row[0], b = row[1];
        const float w = weights[t * k + s];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = fmaf(w, a[e], v[e]);
            v[4 + e] = fmaf(w, b[e], v[4 + e]);
        }
    }
    *reinterpret_cast<u32x4*>(out + t * R + r) = u32x4{pack_x16<H>(v[0], v[1]), pack_x16<H>(v[2], v[3]), pack_x16<H>(v[4], v[5]), pack_x16<H>(v[6], v[7])};
}

template <bool GATED, int OUT>
hipError_t launch_tiles(const Tiling& t, const TileArgs& p, hipStream_t st)
{
    const dim3 grid((unsigned)(8 * cdiv(t.na * t.nb, 8))), block((unsigned)t.threads);
    switch (t.shape) {
        case kSkinny16: hipLaunchKernelGGL((skinny_kernel<GATED, OUT, 1>), grid, block, 0, st, p); break;
        case kSkinny32: hipLaunchKernelGGL((skinny_kernel<GATED, OUT, 2>), grid, block, 0, st, p); break;
        case kSkinny64: hipLaunchKernelGGL((skinny_kernel<GATED, OUT, 4>), grid, block, 0, st, p); break;
        case kSmall: hipLaunchKernelGGL((tile_kernel<GATED, OUT, 2, 2, 4, 4>), grid, block, 0, st, p); break;
        default: hipLaunchKernelGGL((tile_kernel<GATED, OUT, 2, 4, 8, 4>), grid, block, 0, st, p); break;
    }
    return hipGetLastError();
}

}  // namespace

int launch_products(const Geometry& g, const Args& a, void* stream)
{
    clear_pending_error();
    hipStream_t st = (hipStream_t)stream;
    const Tiling t = make_tiling(g);
    const TileArgs p = {a, g.P, g.E, g.R, g.act, (uint32_t)g.kb(), (uint32_t)g.sb(), (uint32_t)t.na, (uint32_t)g.share, (uint32_t)g.X};
    if (g.op == kGlu) return (int)(g.f16 ? launch_tiles<true, kOutF16>(t, p, st) : launch_tiles<true, kOutBf16>(t, p, st));
    if (g.op == kProduct) return (int)(g.f16 ? launch_tiles<false, kOutF16>(t, p, st) : launch_tiles<false, kOutBf16>(t, p, st));
    hipError_t e = launch_tiles<false, kOutF32>(t, p, st);
    if (e != hipSuccess) return (int)e;
    const int64_t T = g.P / a.top_k;
    const dim3 grid((unsigned)cdiv(T * (g.R / 8), 256));
    if (g.f16) hipLaunchKernelGGL(combine_kernel<true>, grid, dim3(256), 0, st, a.part, a.weights, static_cast<uint16_t*>(a.out), T, (int)a.top_k, g.R);
    else hipLaunchKernelGGL(combine_kernel<false>, grid, dim3(256), 0, st, a.part, a.weights, static_cast<uint16_t*>(a.out), T, (int)a.top_k, g.R);
    return (int)hipGetLastError();
}

}  // namespace experts
}  // namespace mhc
