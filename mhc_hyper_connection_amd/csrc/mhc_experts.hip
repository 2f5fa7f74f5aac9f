// mhc_experts.hip -- gfx950 kernels of the products with 4-bit weights.
//
//   product       y = x w^T
//   experts_glu   h[p] = act(x[p / k] Wg[e]^T) (.) (x[p / k] Wu[e]^T)   for the pairs p of each expert e
//   experts_down  y[t] = sum_j weights[t, j] (h[t, j] Wd[e]^T)
// x, h and the weights are microscaled 4-bit floats (mhc_mxfp4_device.h); the matrix instruction takes
// codes and scale bytes as they are in memory: a lane's 16 bytes of codes are one block of 32
// values, and its scale byte that block's. Products accumulate in fp32; the activation and the
// weighted sum are fp32, one rounding to the 16-bit result.
// The weighted sum is a pass of its own over the pairs' results, which wait in the workspace in fp32. Where the caller allows it
// (MHC_SHORT_TERMS), those of bf16 tiles wait as fp16 with a power of two for each 32 of a pair, by which the largest finite one
// is in [2^14, 2^15). That keeps 11 significant bits down to 2^-28 of the largest, three more than the sum's result has, and
// halves what is written and read again: 823 against 634 us a call (65536 pairs, D = 4096, F = 2048). The results differ by 8.9e-4 of their
// norm, some by a bf16 step, and their distance from 64 bits is 1.673e-3 of the norm instead of 1.660e-3. fp16 results, which
// have 11 bits themselves, and the streaming kernel's always wait in fp32.
//
// A unit of work is a run of weight rows and up to a tile's columns of one expert's pairs, which are
// gathered by the plan's list as their x rows are loaded. Pairs without an expert are a bucket of their own
// behind the last expert's: their results are zeros.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "mhc_experts_plan.h"
#include "mhc_mxfp4_device.h"
#include "mhc_tile_device.h"

namespace mhc {
namespace experts {
namespace {

enum Out { kOutBf16, kOutF16, kOutF32, kOutPart };

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

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

// wait_loads_and_barrier<0>, without the wait for memory where m is 0. In one piece: a branch that the compiler sees
// would split the loop's body, and the registers would no longer do.
__device__ __forceinline__ void wait_unless_zero_and_barrier(int m)
{
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_cmp_eq_u32 %0, 0\n\ts_cbranch_scc1 .Lmeet%=\n\ts_waitcnt vmcnt(0)\n.Lmeet%=:\n\ts_barrier" : : "s"(m) : "scc", "memory");
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
    int K, cols, f16;      // cols: of a streaming unit; f16: x's format
};

// A unit: of expert e the units' row a and the pairs [first, first + cols). An XCD (workgroups b, b + 8, ..) takes a
// contiguous run of the units, each of its workgroups every so many of them. The experts' buckets are counted from the plan's
// offsets, which are bounded here: whatever they hold, pairs stay in [0, P).
struct Unit {
    int e;
    uint32_t a;
    int64_t first;
    int cols;
};
// The same in every lane: to a scalar register, which the direct loads' descriptors have to be in.
__device__ __forceinline__ int scalar(int x)
{
    int s;
    asm volatile("s_nop 1\n\tv_readfirstlane_b32 %0, %1" : "=s"(s) : "v"(x));
    return s;
}
// A bucket's first and last pair and its units of BC pairs; bucket E: the pairs without an expert.
__device__ __forceinline__ int bucket(const TileArgs& p, int BC, int e, int* begin, int* end)
{
    bucket_pairs(p.t.offsets, p.E, (int)p.P, e, begin, end);
    return (int)(((int64_t)*end - *begin + BC - 1) / BC);
}
__device__ __forceinline__ uint32_t count_units(const TileArgs& p, int BC)   // along the pairs
{
    if (!p.t.offsets) return (uint32_t)((p.P + BC - 1) / BC);
    const int lane = threadIdx.x & 63, most = most_units(p.P, BC, p.E);
    int total = 0;
    for (int e0 = 0; e0 <= p.E; e0 += 64) {
        int begin, end, n = bucket(p, BC, e0 + lane, &begin, &end);
#pragma unroll
        for (int d = 1; d < 64; d *= 2) n += __shfl_xor(n, d);
        total = units_sum(total, __builtin_amdgcn_readfirstlane(n), most);
    }
    return (uint32_t)total;
}
// Unit i of this XCD's (the streaming kernel's), of total x na in all; false past the last.
__device__ __forceinline__ bool unit_of(const TileArgs& p, int BC, uint32_t total, uint32_t i, Unit* u)
{
    const int lane = threadIdx.x & 63;
    const uint32_t units = total * p.na, per = (units + 7) / 8, unit = blockIdx.x % 8 * per + i;
    if (i >= per || unit >= units) return false;
    uint32_t a = 0, b = 0;
    int e = 0, b0 = 0, b1 = (int)p.P;
    if (!p.t.offsets) place(unit, p.na, total, &a, &b);
    else {
        const uint32_t q = unit / p.na;
        uint32_t at = 0;
        for (int e0 = 0; e0 <= p.E; e0 += 64) {
            int begin, end;
            const int n = bucket(p, BC, e0 + lane, &begin, &end);
            int scan = n;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const int o = __shfl_up(scan, d);
                if (lane >= d) scan += o;
            }
            const uint64_t past = __ballot(q < at + (uint32_t)scan);
            if (past) {
                const int l = __builtin_ctzll(past);
                const uint32_t nb = (uint32_t)__builtin_amdgcn_readlane(n, l);
                at += (uint32_t)(__builtin_amdgcn_readlane(scan, l) - (int)nb);
                b0 = __builtin_amdgcn_readlane(begin, l);
                b1 = __builtin_amdgcn_readlane(end, l);
                place(unit - at * p.na, p.na, nb, &a, &b);
                e = e0 + l;
                break;
            }
            at += (uint32_t)__builtin_amdgcn_readlane(scan, 63);
        }
    }
    const int64_t first = b0 + (int64_t)b * BC;
    u->e = scalar(e);
    u->a = (uint32_t)scalar((int)a);
    u->first = (int64_t)(uint32_t)scalar((int)first);    // under 2^31
    u->cols = scalar((int)(b1 - first < BC ? b1 - first : BC));
    return true;
}
// The units of a tiled workgroup, lane n's the n-th (at most 64: the plan sees to it), found before its first loads: a search
// between two units took 4 us, in which nothing was multiplied. `lds` holds the buckets' beginnings meanwhile.
struct Units {
    uint32_t place;        // e, a and cols - 1 in 11, 10 and 8 bits
    int first;             // -1: no such unit
    __device__ __forceinline__ bool at(int n, Unit* u) const
    {
        const uint32_t w = (uint32_t)__builtin_amdgcn_readlane((int)place, n);
        const int f = __builtin_amdgcn_readlane(first, n);
        u->e = (int)(w & 0x7ff);
        u->a = (w >> 11) & 0x3ff;
        u->cols = (int)(w >> 21) + 1;
        u->first = f;
        return f >= 0;
    }
};
constexpr int kUnitsLds = 3 * (kMaxE + 2) * 4;
template <int BC>
__device__ __forceinline__ Units units_of(const TileArgs& p, int* lds)
{
    const int lane = threadIdx.x & 63;
    int* const before = lds;                       // units along the pairs before a bucket's
    int* const begin = lds + kMaxE + 2;
    int* const end = begin + kMaxE + 2;
    uint32_t total = (uint32_t)((p.P + BC - 1) / BC);
    if (p.t.offsets) {
        if (threadIdx.x < 64) {
            const int most = most_units(p.P, BC, p.E);
            int at = 0;
            for (int e0 = 0; e0 <= p.E; e0 += 64) {
                int b, n;
                const int tiles = bucket(p, BC, e0 + lane, &b, &n);
                int scan = tiles;
#pragma unroll
                for (int d = 1; d < 64; d *= 2) {
                    const int o = __shfl_up(scan, d);
                    if (lane >= d) scan += o;
                }
                if (e0 + lane <= p.E) {
                    before[e0 + lane] = units_sum(at, scan - tiles, most);
                    begin[e0 + lane] = b;
                    end[e0 + lane] = n;
                }
                at = units_sum(at, __builtin_amdgcn_readlane(scan, 63), most);
            }
            if (lane == 0) before[p.E + 1] = at;
        }
        __syncthreads();
        total = (uint32_t)before[p.E + 1];
    }
    const uint32_t units = total * p.na, per = (units + 7) / 8, i = blockIdx.x / 8 + (uint32_t)lane * (gridDim.x / 8), unit = blockIdx.x % 8 * per + i;
    Units u = {0, -1};
    if (i < per && unit < units) {
        uint32_t a, b;
        int e = 0, b0 = 0, b1 = (int)p.P;
        int64_t first;
        if (p.t.offsets) {
            find_unit(before, begin, p.E, p.na, BC, unit, &e, &a, &first);
            b0 = begin[e];
            b1 = end[e];
        } else {
            place(unit, p.na, total, &a, &b);
            first = (int64_t)b * BC;
        }
        if (first >= b0 && first < b1) {           // of a plan's offsets always
            u.first = (int)first;
            u.place = (uint32_t)e | a << 11 | (uint32_t)((b1 - first < BC ? (int)(b1 - first) : BC) - 1) << 21;
        }
    }
    __syncthreads();
    return u;
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
            *reinterpret_cast<f32x4*>(static_cast<float*>(p.t.part) + pair * p.R + r + 4 * h) = f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
    } else {
        uint16_t* const out = static_cast<uint16_t*>(p.t.out) + pair * p.R + r;
        uint32_t w[N / 2];
#pragma unroll
        for (int e = 0; e < N / 2; ++e) w[e] = pack_x16<OUT == kOutF16>(v[2 * e], v[2 * e + 1]);
        if constexpr (N == 8) *reinterpret_cast<u32x4*>(out) = u32x4{w[0], w[1], w[2], w[3]};
        else *reinterpret_cast<u32x2*>(out) = u32x2{w[0], w[1]};
    }
}

// The exponent field of the largest finite magnitude among 32 results of a column, eight in each of four lanes 16 apart; at least
// 15, so that the powers of two below are normal numbers. An infinity or a NaN has no part in it: under any of those
// powers it stays what it is, and a neighbour's is that of the finite ones.
__device__ __forceinline__ uint32_t exponent_of(f32x4 a, f32x4 b)
{
    // as whole numbers, which order like the values; twice them (without the sign) plus one in the exponent: 255 becomes 0
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t x = (__float_as_uint(a[e]) << 1) + 0x01000000u, y = (__float_as_uint(b[e]) << 1) + 0x01000000u;
        m = m > x ? m : x;
        m = m > y ? m : y;
    }
    const auto s = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    m = s[0] > s[1] ? s[0] : s[1];
    const auto t = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    m = (t[0] > t[1] ? t[0] : t[1]) >> 24;
    return (m < 16 ? 16 : m) - 1;
}
// The power of two that takes such results to [2^14, 2^15), and back.
__device__ __forceinline__ uint32_t part_up(uint32_t exponent) { return (268u - exponent) << 23; }
__device__ __forceinline__ uint32_t part_down(uint32_t exponent) { return (exponent - 14u) << 23; }

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
// Loads past the end of the reduction bring zeros. T = 16384, K = 4096, N = 16384: 554 us, 4.0 PFLOP/s; a stage takes 1.7 to
// 1.9 us, of which its products alone would take 1.2: the matrix cores are busy 47 % of the cycles, and the waves in a wait for
// 30 % (for the middle's loads and each other).
template <bool GATED, int OUT, int WA, int WB, int IA, int IB>
__global__ void __launch_bounds__(64 * WA * WB, 2)
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

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wa = wave / WB, wb = wave % WB;
    const int j = lane & 15, kg = lane >> 4;
    const uint32_t kb = p.kb, sb = p.sb;
    const int64_t R = p.R;
    constexpr int ROWS = GATED ? AR / 2 : AR;                    // of one weight
    const u32x4 dxc = descriptor(p.t.x_codes, p.x_rows * kb), dxs = descriptor(p.t.x_scales, p.x_rows * sb);
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>(lds));

    // --- loads of codes, 1 KiB each: 8 LDS rows of 128 bytes. A lane group kg takes the blocks 2 kg and 2 kg + 1 of a
    // stage, one in each half, so that their scales are neighbours; the 16-byte chunk c of row r sits at c ^ s(r), where with
    // the reading lane's number j of 16, s has the bits (j >> 3 ^ j >> 2, j >> 1, j >> 2): each of the four turns of a 16-byte
    // read (the first of lanes 0-3, 12-15 and 20-27) then meets all banks once.
    auto swizzle = [](int j) __attribute__((always_inline)) { return (((j >> 3) ^ (j >> 2)) & 1) * 4 + (j & 2) + ((j >> 2) & 1); };
    // the weight rows of a pair of results are 8 (j / 4) + 4 h + j % 4
    const int r0 = 8 * wave + lane / 8;                      // this lane's row of a wave's first load; the others' have the same swizzle
    const uint32_t ka = 16 * ((lane & 7) ^ swizzle(((r0 >> 1) & 12) + (r0 & 3))), kx = 16 * ((lane & 7) ^ swizzle(r0 & 15));
    static_assert(NW % 4 == 0 && ROWS % (8 * NW) == 0, "rows 32 apart, and a load within one weight");
    // scales, 8 rows of 8 words a load; the pair of words of a row's stage n of 4 sits at n ^ (r / 8) % 4, so that the
    // rows of a block of results, 8 apart or 16 in a run, meet different banks
    const uint32_t ks = 4 * ((lane & 7) ^ (2 * (wave & 3)));
    // where a unit's loads begin
    struct Loads {
        u32x4 dc0, dc1, ds0, ds1;
        uint32_t vb[QB], vs[SB];
    };
    const uint32_t va = (uint32_t)r0 * kb + ka, vsa = (uint32_t)r0 * sb + ks;
    static_assert(SB == QB && SA == QA, "a load of scales has the rows of one of codes");
    // ln: the lane, hidden from the compiler, which would keep all that follows from it through the products
    auto set_up = [=](int ln, const Unit& u, Loads& l) __attribute__((always_inline)) {
        const int64_t a0 = (int64_t)u.a * ROWS, w0 = u.e * R + a0;
        const uint32_t arow = (uint32_t)(R - a0 < ROWS ? R - a0 : ROWS);
        l.dc0 = descriptor(p.t.w_codes[0] + w0 * kb, arow * kb);
        l.dc1 = GATED ? descriptor(p.t.w_codes[1] + w0 * kb, arow * kb) : l.dc0;
        l.ds0 = descriptor(p.t.w_scales[0] + w0 * sb, arow * sb);
        l.ds1 = GATED ? descriptor(p.t.w_scales[1] + w0 * sb, arow * sb) : l.ds0;
        const int r0 = 8 * wave + ln / 8;
        const uint32_t kx = 16 * ((ln & 7) ^ swizzle(r0 & 15));
#pragma unroll
        for (int q = 0; q < QB; ++q) {
            const int64_t pair = pair_of(p, u, r0 + 8 * NW * q);
            const uint32_t x = pair < 0 ? 0u : (uint32_t)pair / p.share;
            l.vb[q] = pair < 0 ? kOutOfRange : x * kb + kx;
            l.vs[q] = pair < 0 ? kOutOfRange : x * sb + ks;
        }
    };
    // where this wave's loads go
    const uint32_t codes_at = (uint32_t)scalar((int)(lds0 + wave * 1024)), scales_at = (uint32_t)scalar((int)(lds0 + 2 * STAGE + wave * 256));
    // hidden anew at each use from the compiler, which would keep the sums with every slot and load, in more registers than there are
    auto hidden = [](uint32_t v) __attribute__((always_inline)) {
        asm volatile("" : "+s"(v));
        return v;
    };
    // load q of this wave's part of a stage of the weights, of the pairs, of either's scales
    auto issue_a = [=](const Loads& l, int step, int slot, int q) __attribute__((always_inline)) {
        const uint32_t k = hidden((uint32_t)step * kLine);
        buffer_to_lds(!GATED || q < QA / 2 ? l.dc0 : l.dc1, k + ka < kb ? va + (k + (8 * NW * q) % ROWS * kb) : kOutOfRange, hidden(codes_at) + slot * STAGE + q * NW * 1024);
    };
    auto issue_b = [=](const Loads& l, int step, int slot, int q) __attribute__((always_inline)) {
        const uint32_t k = hidden((uint32_t)step * kLine);
        buffer_to_lds(dxc, k + kx < kb ? l.vb[q] + k : kOutOfRange, hidden(codes_at) + slot * STAGE + ASZ + q * NW * 1024);
    };
    auto issue_s = [=](const Loads& l, int group, uint32_t slot, int n) __attribute__((always_inline)) {
        const uint32_t s = hidden((uint32_t)group * 32), at = hidden(scales_at) + slot;
        if (n < SA) word_to_lds(!GATED || n < SA / 2 ? l.ds0 : l.ds1, s + ks < sb ? vsa + (s + (8 * NW * n) % ROWS * sb) : kOutOfRange, at + NW * n * 256);
        else word_to_lds(dxs, s + ks < sb ? l.vs[n - SA] + s : kOutOfRange, at + NW * n * 256);
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
    struct Scales {                // of a stage: two bytes, one for each half
        int a[IA], b[IB];
    };
    struct Pairs {                 // those of two blocks of results in a word
        int a[IA / 2], b[IB / 2];
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
        o.a[i] = *(const MHC_LDS uint16_t*)(uintptr_t)((asc ^ (n << 3)) + slot + row_of(i) * 32);
    };
    auto read_sb = [=](uint32_t slot, int n, int q, Scales& o) __attribute__((always_inline)) {
        o.b[q] = *(const MHC_LDS uint16_t*)(uintptr_t)((bsc ^ ((n ^ 2 * (q & 1)) << 3)) + slot + q * 16 * 32);
    };

    // a unit's first loads: its first group of scales and two stages
    auto first_loads = [=](const Loads& l) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < SA + SB; ++n) issue_s(l, 0, 0, n);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int q = 0; q < QA; ++q) issue_a(l, s, s, q);
#pragma unroll
            for (int q = 0; q < QB; ++q) issue_b(l, s, s, q);
        }
    };

    const int steps = (int)((kb + kLine - 1) / kLine);
    static_assert(BC <= 256 && kUnitsLds <= (int)sizeof(lds), "a unit's columns in 8 bits, the buckets where the stages go");
    const Units mine = units_of<BC>(p, reinterpret_cast<int*>(lds));
    int n = 0;
    Unit u, next;
    if (!mine.at(0, &u)) return;
    Loads l;
    if (u.e < p.E) {
        set_up(lane, u, l);
        first_loads(l);
    }
    wait_loads_and_barrier<GATED ? QA + QB : 0>();
    while (true) {
        f32x4 acc[IA][IB];
#pragma unroll
        for (int i = 0; i < IA; ++i)
#pragma unroll
            for (int q = 0; q < IB; ++q) acc[i][q] = f32x4{0.f, 0.f, 0.f, 0.f};
        const bool more = !GATED && ++n < 64 && mine.at(n, &next);

        if (u.e < p.E) {
            Operands op[2];
            Scales sc;
            Pairs sp;
#pragma unroll
            for (int q = 0; q < IB; ++q) read_b(0, 0, q, op[0]), read_sb(0, 0, q, sc);
#pragma unroll
            for (int i = 0; i < IA; ++i) read_a(0, 0, i, op[0]), read_sa(0, 0, i, sc);
            // half H2 of stage m = 4 group + n: the products of `now` in IA parts, the reads of the next half (and of the next
            // stage's scales) and the loads dealt out over them; `slot`: where the next stage's scales are, `other`: the next group's
            auto half = [&](auto number, int m, int n, const Operands& now, Operands& next, uint32_t slot,
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
                            if (H2) read_sb(slot, (n + 1) % 4, r, sc);
                        } else {
                            read_a(rs, 1 - H2, r - IB, next);
                            if (H2) read_sa(slot, (n + 1) % 4, r - IB, sc);
                        }
                    }
                    if (!H2) {     // the scales read in the half before
                        if (i % 2 == 0) sp.a[i / 2] = sc.a[i] | sc.a[i + 1] << 16;
#pragma unroll
                        for (int q = 0; q < (i == 0 ? IB : 0); q += 2) sp.b[q / 2] = sc.b[q] | sc.b[q + 1] << 16;
                    }
                    const int sa = sp.a[i / 2];
#pragma unroll
                    for (int q = 0; q < IB; ++q) {
                        const int sb2 = sp.b[q / 2];
                        f32x4& c = acc[i][q];
                        if (i % 2 == 0) c = q % 2 == 0 ? mfma4<H2, H2>(now.a[i], now.b[q], c, sa, sb2) : mfma4<H2, 2 + H2>(now.a[i], now.b[q], c, sa, sb2);
                        else c = q % 2 == 0 ? mfma4<2 + H2, H2>(now.a[i], now.b[q], c, sa, sb2) : mfma4<2 + H2, 2 + H2>(now.a[i], now.b[q], c, sa, sb2);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    if (H2 == 1) {
#pragma unroll
                        for (int q = i * QA / IA; q < (i + 1) * QA / IA; ++q) issue_a(l, m + 2, s, q);
#pragma unroll
                        for (int q = i * QB / IA; q < (i + 1) * QB / IA; ++q) issue_b(l, m + 2, s, q);
#pragma unroll
                        for (int q = i * QN / IA; q < (i + 1) * QN / IA; ++q) issue_s(l, m / 4 + 1, other, n * (SA + SB) / 3 + q);
                    }
                }
            };
            uint32_t slot = 0;
            for (int m = 0; m < steps; m += 4) {
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    if (m + n < steps) {
                        half(Number<0>{}, m + n, n, op[0], op[1], slot, slot ^ GROUP);
                        // stage 1 is there from before; the last unit's stores may still be on their way
                        if (!GATED && n == 0) wait_unless_zero_and_barrier(m);
                        else wait_loads_and_barrier<0>();
                        half(Number<1>{}, m + n, n, op[1], op[0], n == 3 ? slot ^ GROUP : slot, slot ^ GROUP);
                    }
                }
                slot ^= GROUP;
            }
            wait_loads_and_barrier<0>();   // no load is left behind in LDS, and every wave has read it
        }

        // --- results: lane (j, kg) holds rows 4 kg .. 4 kg + 3 of column j of each 16 x 16 block: 8 kg .. 8 kg + 7 of the 32 rows of
        // a pair of blocks
        const int64_t a0 = (int64_t)u.a * ROWS + wa * WR;        // the wave's first row
        int ln = lane;
        asm volatile("" : "+v"(ln));
        if constexpr (GATED) {
            auto results = [&](auto act) __attribute__((always_inline)) {
#pragma unroll
                for (int q = 0; q < IB; ++q) {
                    const int64_t pair = pair_of(p, u, 16 * (wb * IB + q) + j);
#pragma unroll
                    for (int i = 0; i < IA / 4; ++i) {
                        const int64_t f = a0 + 32 * i + 8 * kg;
                        float v[8];
#pragma unroll
                        for (int r = 0; r < 8; ++r)
                            v[r] = activation<decltype(act)::value>(acc[2 * i + r / 4][q][r % 4]).a * acc[IA / 2 + 2 * i + r / 4][q][r % 4];
                        if (pair >= 0 && f < R) store_results<OUT>(p, pair, f, v);
                    }
                }
            };
            if (p.act) results(Number<1>{});
            else results(Number<0>{});
            return;
        }
        // A store takes eight neighbouring lanes to a column, whose 16-byte pieces are a whole line of memory (of two runs of 32
        // 16-bit results, or one of fp32); stored from where they are, 16 lanes apart and half a line at a time, they took longer:
        // 592 against 571 us for T = 16384, K = 4096, N = 16384, and 634 through the caches. (The gated projection's stores go out
        // between the activations, and gain nothing by it.)
        auto from = [](int lane4, uint32_t v) __attribute__((always_inline)) { return (uint32_t)__builtin_amdgcn_ds_bpermute(lane4, (int)v); };
        // columns 8 c .. of a block of 16: piece ln % 8 of column ln / 8, of run 0 (w) or 1 (v) of the two
        auto line = [=](int c, const uint32_t (&w)[4], const uint32_t (&v)[4]) __attribute__((always_inline)) {
            const int src = 4 * (8 * c + ln / 8 + 16 * (ln & 3));
            u32x4 o;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t x = from(src, w[e]), y = from(src, v[e]);
                o[e] = ln & 4 ? y : x;
            }
            return o;
        };
        // They are stored once the next unit's first loads are there, and are on their way while its first stages are multiplied.
        if (more && next.e < p.E) {
            set_up(ln, next, l);
            first_loads(l);
        }
        int pair[IB][2];
#pragma unroll
        for (int q = 0; q < IB; ++q)
#pragma unroll
            for (int c = 0; c < 2; ++c) pair[q][c] = (int)pair_of(p, u, 16 * (wb * IB + q) + 8 * c + ln / 8);
        wait_loads_and_barrier<0>();
        const int64_t RS = part_scales(R);
#pragma unroll
        for (int q = 0; q < IB; ++q) {
            uint32_t exponent = 0;       // of run kg
#pragma unroll
            for (int i = 0; i < IA / 2; ++i) {
                if constexpr (OUT == kOutF32) {
                    const int64_t f = a0 + 32 * i + 4 * (ln & 7);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int src = 4 * (8 * c + ln / 8 + 16 * ((ln & 7) >> 1));
                        u32x4 w;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t lo = from(src, __float_as_uint(acc[2 * i][q][e])), hi = from(src, __float_as_uint(acc[2 * i + 1][q][e]));
                            w[e] = ln & 1 ? hi : lo;
                        }
                        if (pair[q][c] >= 0 && f < R) __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(static_cast<float*>(p.t.part) + (int64_t)pair[q][c] * R + f));
                    }
                } else if (i % 2 == 0) {
                    float scale[2] = {1.f, 1.f};
                    if constexpr (OUT == kOutPart) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t e = exponent_of(acc[2 * i + 2 * h][q], acc[2 * i + 2 * h + 1][q]);
                            scale[h] = __uint_as_float(part_up(e));
                            exponent = (ln >> 4) == i + h ? e : exponent;
                        }
                    }
                    uint32_t w[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float lo = acc[2 * i + 2 * h + e / 2][q][2 * (e % 2)], hi = acc[2 * i + 2 * h + e / 2][q][2 * (e % 2) + 1];
                            w[h][e] = OUT == kOutPart ? pack_f16x2(lo * scale[h], hi * scale[h]) : pack_x16<OUT == kOutF16>(lo, hi);
                        }
                    const int64_t f = a0 + 32 * i + 8 * (ln & 7);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const u32x4 o = line(c, w[0], w[1]);
                        if (pair[q][c] >= 0 && f < R)
                            __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(OUT == kOutPart ? p.t.part : p.t.out) + (int64_t)pair[q][c] * R + f));
                    }
                }
            }
            if constexpr (OUT == kOutPart) {
                // a byte for each run of the wave's
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint32_t e = from(4 * (8 * c + ln / 8 + 16 * (ln & 3)), exponent);
                    const int64_t run = a0 / 32 + (ln & 3);
                    if (pair[q][c] >= 0 && (ln & 7) < IA / 2 && run < RS) p.t.part_scales[(int64_t)pair[q][c] * RS + run] = (uint8_t)e;
                }
            }
        }
        if (!more) break;
        u = next;
    }
}

// Few pairs of an expert (16 at most to a unit): reading the weights once is the whole cost. A
// workgroup takes 32 weight rows (gated: 16 of either weight), its W waves every W-th stage of 256 values; their
// sums meet in LDS and are added in wave order. A wave keeps a ring of three stages of its own in LDS,
// so that it waits for its own loads only and meets the others once. K = 7168, N = 16384, one token: 13.3 us for 62 MB of weights;
// 64 experts, top 8, D = 7168, F = 2048, gated: 25.5 for 125 MB: 4.7 and 4.9 TB/s, with some 2 us to start and to join. X16: the
// pairs' x rows come in 16 bits and are rounded into LDS, behind the first loads of weights, once for all their stages.
template <bool GATED, int OUT, bool X16>
__global__ void __launch_bounds__(256)
skinny_kernel(TileArgs p)
{
    constexpr int W = 4, RING = 3, ROWS = X16 ? 32 : 32 + 16;
    // loads of scales: 32 rows of a weight, or 16 of either of two; 16 of the pairs (half a load, the other lanes idle)
    constexpr int SW = GATED ? 2 : 1;
    constexpr int CODES = ROWS * kLine, STAGE = CODES + ROWS * 8, LOADS = ROWS / 8 + SW + (X16 ? 0 : 1);
    static_assert(RING * STAGE >= 2 * 64 * 16, "a wave's sums fit where its stages were");
    static_assert(!X16 || W * RING * STAGE + kRoundedX == 81920, "half of the LDS");
    __shared__ __attribute__((aligned(1024))) char lds[X16 ? 81920 : W * RING * STAGE];
    Unit u;
    if (!unit_of(p, p.cols, count_units(p, p.cols), blockIdx.x / 8, &u)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15, kg = lane >> 4;
    const uint32_t kb = p.kb, sb = p.sb;
    constexpr int WR = GATED ? 16 : 32;                          // rows of one weight
    const int64_t a0 = (int64_t)u.a * WR, R = p.R;
    const uint32_t arow = (uint32_t)(R - a0 < WR ? R - a0 : WR);

    f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
    if (u.e < p.E) {
        const int64_t w0 = u.e * R + a0;
        const u32x4 dc0 = descriptor(p.t.w_codes[0] + w0 * kb, arow * kb), ds0 = descriptor(p.t.w_scales[0] + w0 * sb, arow * sb);
        const u32x4 dc1 = GATED ? descriptor(p.t.w_codes[1] + w0 * kb, arow * kb) : dc0;
        const u32x4 ds1 = GATED ? descriptor(p.t.w_scales[1] + w0 * sb, arow * sb) : ds0;
        const u32x4 dxc = descriptor(p.t.x_codes, X16 ? 0 : p.x_rows * kb), dxs = descriptor(p.t.x_scales, X16 ? 0 : p.x_rows * sb);
        const uint32_t mine = __builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>(lds)) + wave * (RING * STAGE);
        // a load of codes takes 8 rows; chunk c of row r sits at c ^ (r / 2) % 8
        const int lr = lane / 8, lc = lane & 7;
        uint32_t vx[2] = {0, 0}, kx[2] = {0, 0}, vs = 0;
        if constexpr (!X16) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 8 * i + lr, c = lc ^ ((r >> 1) & 7);
                const int64_t q = pair_of(p, u, r);
                kx[i] = 16 * c;
                vx[i] = q < 0 ? kOutOfRange : ((uint32_t)q / p.share) * kb + kx[i];
            }
            {
                const int64_t q = pair_of(p, u, lane / 2);           // lanes past 16 rows are idle
                vs = q < 0 ? kOutOfRange : ((uint32_t)q / p.share) * sb;
            }
        }
        auto issue = [=](int step, int slot) __attribute__((always_inline)) {
            const uint32_t k = (uint32_t)step * kLine, s = (uint32_t)step * 8, at = mine + slot * STAGE;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 8 * (GATED ? i % 2 : i) + lr, c = lc ^ ((r >> 1) & 7);
                buffer_to_lds(GATED && i >= 2 ? dc1 : dc0, k + 16 * c < kb ? (uint32_t)r * kb + k + 16 * c : kOutOfRange, at + i * 1024);
            }
#pragma unroll
            for (int i = 0; i < (X16 ? 0 : 2); ++i)
                buffer_to_lds(dxc, k + kx[i] < kb ? vx[i] + k : kOutOfRange, at + (4 + i) * 1024);
            const uint32_t w = s + 4 * (lane & 1);               // rows past the weight's are out of range
#pragma unroll
            for (int i = 0; i < SW; ++i)
                if (!GATED || lane < 32)
                    word_to_lds(i ? ds1 : ds0, w < sb ? (uint32_t)(lane / 2) * sb + w : kOutOfRange, at + CODES + i * 128);
            if (!X16 && lane < 32) word_to_lds(dxs, w < sb ? vs + w : kOutOfRange, at + CODES + 256);
        };
        const uint32_t at0 = mine + j * kLine + ((kg ^ (j >> 1)) << 4), sc0 = mine + CODES + j * 8 + kg;
        const int steps = (int)((kb + kLine - 1) / kLine);
#pragma unroll
        for (int s = 0; s < RING - 1; ++s) issue(wave + s * W, s);
        // the rounded rows: of each column the codes of all stages, then their scales
        char* const rounded = lds + W * RING * STAGE;
        if constexpr (X16) {
            const int octets = steps * 32, row = (int)rounded_row(steps);
            for (int i = tid; i < u.cols * octets; i += 64 * W) {
                const int c = i / octets, o = i - c * octets;    // four lanes share a block
                const int64_t q = pair_of(p, u, c);
                u32x4 v = {0u, 0u, 0u, 0u};
                if (q >= 0) {
                    const uint16_t* const at = p.t.x + (int64_t)((uint32_t)q / p.share) * p.K + 8 * o;
                    if (p.K % 8 == 0) {
                        if (8 * o < p.K) v = *reinterpret_cast<const u32x4*>(at);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (8 * o + e < p.K) v[e / 2] |= (uint32_t)at[e] << (16 * (e & 1));
                    }
                }
                uint32_t m = mx_absmax(v);
                m = mx_dpp_max<kQuadXor2>(mx_dpp_max<kQuadXor1>(m));
                const uint32_t scale = p.f16 ? mx_scale<true>(m) : mx_scale<false>(m);
                *reinterpret_cast<uint32_t*>(rounded + c * row + 4 * o) = p.f16 ? mx_encode<true>(v, scale) : mx_encode<false>(v, scale);
                if ((o & 3) == 0) rounded[c * row + steps * 128 + o / 4] = (char)scale;
            }
            __syncthreads();
        }
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
                        i32x4 x = {0, 0, 0, 0};
                        int sx = 0;
                        if constexpr (X16) {
                            const char* const r = rounded + j * (int)rounded_row(steps);
                            const int block = (k + s * W) * 8 + 4 * h + kg;
                            if (j < u.cols) {
                                x = *reinterpret_cast<const i32x4*>(r + 16 * block);
                                sx = *reinterpret_cast<const uint8_t*>(r + steps * 128 + block);
                            }
                        } else {
                            x = *(const MHC_LDS i32x4*)(uintptr_t)(at + 32 * kLine);
                            sx = *(const MHC_LDS uint8_t*)(uintptr_t)(sc + 256);
                        }
                        acc[0] = mfma4<0, 0>(w0v, x, acc[0], s0, sx);
                        acc[1] = mfma4<0, 0>(w1v, x, acc[1], s1, sx);
                    }
                    asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");   // read, before the slot is loaded again
                }
            }
        }
        asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
    }
    // the sums, each wave's where its stages were
    auto red = [&](int w, int i) { return reinterpret_cast<f32x4*>(lds + w * (RING * STAGE)) + i * 64; };
    red(wave, 0)[lane] = acc[0];
    red(wave, 1)[lane] = acc[1];
    __syncthreads();
    if (wave > 0) return;
    f32x4 v0 = red(0, 0)[lane], v1 = red(0, 1)[lane];
#pragma unroll
    for (int w = 1; w < W; ++w) {
        v0 += red(w, 0)[lane];
        v1 += red(w, 1)[lane];
    }
    const int64_t pair = pair_of(p, u, j), r = a0 + 4 * kg;
    if (pair < 0) return;
    if constexpr (GATED) {
        float v[4];
        if (p.act) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = activation<1>(v0[e]).a * v1[e];
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = activation<0>(v0[e]).a * v1[e];
        }
        if (r < R) store_results<OUT>(p, pair, r, v);
    } else {
        const float lo[4] = {v0[0], v0[1], v0[2], v0[3]}, hi[4] = {v1[0], v1[1], v1[2], v1[3]};
        if (r < R) store_results<OUT>(p, pair, r, lo);
        if (r + 16 < R) store_results<OUT>(p, pair, r + 16, hi);
    }
}

// A token's results by its weights: fp32 terms in the order of its slots, one rounding. A thread takes eight values. HBM bounds it:
// 8192 tokens of 8 slots, D = 4096, 1.14 GB in 210 us, 5.4 TB/s; PART, terms in 16 bits: 604 MB in 100 us, 6.0 TB/s.
template <bool H, bool PART>
__global__ void __launch_bounds__(256)
combine_kernel(const void* __restrict__ part, const uint8_t* __restrict__ scales, const float* __restrict__ weights, uint16_t* __restrict__ out, int64_t T, int k,
               int R)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int octets = R / 8;
    const int64_t t = i / octets;
    if (t >= T) return;
    const int64_t r = (i - t * octets) * 8;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = 0; s < k; ++s) {
        const int64_t row = t * k + s;
        const float w = weights[row];
        if constexpr (PART) {
            const u32x4 a = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(part) + row * R + r));
            const float x = __uint_as_float(part_down(scales[row * part_scales(R) + r / 32]));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[2 * e] = fmaf(w, f16_lo(a[e]) * x, v[2 * e]);
                v[2 * e + 1] = fmaf(w, f16_hi(a[e]) * x, v[2 * e + 1]);
            }
        } else {
            const f32x4* const at = reinterpret_cast<const f32x4*>(static_cast<const float*>(part) + row * R + r);
            const f32x4 a = at[0], b = at[1];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = fmaf(w, a[e], v[e]);
                v[4 + e] = fmaf(w, b[e], v[4 + e]);
            }
        }
    }
    *reinterpret_cast<u32x4*>(out + t * R + r) = u32x4{pack_x16<H>(v[0], v[1]), pack_x16<H>(v[2], v[3]), pack_x16<H>(v[4], v[5]), pack_x16<H>(v[6], v[7])};
}

template <bool GATED, int OUT>
hipError_t launch_tiles(const Tiling& t, const TileArgs& p, hipStream_t st)
{
    const dim3 grid((unsigned)t.grid()), block((unsigned)t.threads);
    switch (t.shape) {
        case kSkinny:
            if constexpr (OUT != kOutPart) {
                if (t.rounds_x) hipLaunchKernelGGL((skinny_kernel<GATED, OUT, true>), grid, block, 0, st, p);
                else hipLaunchKernelGGL((skinny_kernel<GATED, OUT, false>), grid, block, 0, st, p);
            }
            break;
        case kSmall: hipLaunchKernelGGL((tile_kernel<GATED, OUT, 2, 2, 4, 4>), grid, block, 0, st, p); break;
        default: hipLaunchKernelGGL((tile_kernel<GATED, OUT, 2, 4, 8, 4>), grid, block, 0, st, p); break;
    }
    return hipGetLastError();
}

}  // namespace

int launch_products(const Geometry& g, const Tiling& t, const Args& a, void* stream)
{
    clear_pending_error();
    hipStream_t st = (hipStream_t)stream;
    const TileArgs p = {a, g.P, g.E, g.R, g.act, (uint32_t)g.kb(), (uint32_t)g.sb(), (uint32_t)t.na, (uint32_t)g.share, (uint32_t)g.X,
                        g.K, t.cols, g.f16};
    if (g.op == kGlu) return (int)(g.f16 ? launch_tiles<true, kOutF16>(t, p, st) : launch_tiles<true, kOutBf16>(t, p, st));
    if (g.op == kProduct) return (int)(g.f16 ? launch_tiles<false, kOutF16>(t, p, st) : launch_tiles<false, kOutBf16>(t, p, st));
    const bool in16 = parts_in_16_bits(g);
    const hipError_t e = in16 ? launch_tiles<false, kOutPart>(t, p, st) : launch_tiles<false, kOutF32>(t, p, st);
    if (e != hipSuccess) return (int)e;
    const int64_t T = g.P / a.top_k;
    const dim3 grid((unsigned)cdiv(T * (g.R / 8), 256)), block(256);
    uint16_t* const out = static_cast<uint16_t*>(a.out);
    const int k = (int)a.top_k;
    if (in16) hipLaunchKernelGGL((combine_kernel<false, true>), grid, block, 0, st, a.part, a.part_scales, a.weights, out, T, k, g.R);
    else if (g.f16) hipLaunchKernelGGL((combine_kernel<true, false>), grid, block, 0, st, a.part, a.part_scales, a.weights, out, T, k, g.R);
    else hipLaunchKernelGGL((combine_kernel<false, false>), grid, block, 0, st, a.part, a.part_scales, a.weights, out, T, k, g.R);
    return (int)hipGetLastError();
}

}  // namespace experts
}  // namespace mhc
