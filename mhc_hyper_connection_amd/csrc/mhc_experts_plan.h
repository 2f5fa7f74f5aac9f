// mhc_experts_plan.h -- geometry, launch shapes and workspace layout of the products with
// 4-bit weights: y = x w^T, the experts' gated projection, and their projection back.
//
// Host-side and plain C++ (no HIP headers), like mhc_plan.h.
#pragma once

#include <cstddef>
#include <cstdint>

#include "mhc_mxfp4_plan.h"

#ifdef __HIP__
#define MHC_EXPERTS_HOST_DEVICE __host__ __device__
#else
#define MHC_EXPERTS_HOST_DEVICE
#endif

namespace mhc {
namespace experts {

constexpr int kMaxE = 1024;
constexpr int kMaxTopK = 32;
constexpr int kMaxDim = 65536;        // D, F, K, N
constexpr int kCUs = 256;

enum Op { kProduct = 0, kGlu = 1, kDown = 2 };

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// P rows of results of R values each over a reduction of K. An x row serves `share` result rows (the
// experts' gated projection: a token's k pairs).
struct Geometry {
    int op = 0;
    int64_t P = 0, X = 0;     // result rows, x rows
    int E = 1, share = 1;
    int K = 0, R = 0;
    int act = 0, f16 = 0;
    int short_terms = 0;      // kDown: the caller allows its terms in 16 bits
    int64_t kb() const { return mx::code_bytes(K); }
    int64_t sb() const { return mx::scale_bytes(K); }
};

// A unit: `rows` weight rows (of the gated projection: of both weights together) and up to `cols`
// pairs of one expert. Few pairs: kSkinny, whose workgroups stream the weights past 16 of them.
enum Shape { kSkinny, kSmall, kLarge };
struct Tiling {
    int shape = kLarge;
    int rows = 256, cols = 256, threads = 512;
    int64_t na = 0;           // units along the weight rows
    int64_t nb = 0;           // units along the pairs, at most: every expert may end in a part of one
    int64_t places = 0;       // workgroups that take the units in turn; 0: one for each
    bool rounds_x = false;    // kSkinny: takes x in 16 bits and rounds it itself
    int64_t grid() const
    {
        const int64_t n = 8 * cdiv(na * nb, 8);
        if (!places || n <= places) return n;
        const int64_t least = 8 * cdiv(n, 8 * 64);       // a workgroup knows 64 of its units
        return places > least ? places : least;
    }
};

// The streaming kernel's LDS beside its rings of weights, for rows of x that it rounds itself.
constexpr int64_t kRoundedX = 81920 - 12 * (32 * 128 + 256);
MHC_EXPERTS_HOST_DEVICE inline int64_t rounded_row(int64_t stages) { return (stages * 136 + 15) / 16 * 16; }      // codes and scales
// How the work is cut; x16: x comes in 16 bits.
inline Tiling make_tiling(const Geometry& g, bool x16 = false)
{
    Tiling t;
    const int64_t rows = g.op == kGlu ? 2 * (int64_t)g.R : g.R, steps = cdiv(g.kb(), 128);
    const int64_t d = g.P < g.E ? g.P : g.E;                     // experts that may have pairs
    // units along the pairs: every expert's last one half full
    auto across = [&](int64_t cols) {
        const int64_t n = g.op == kProduct ? cdiv(g.P, cols) : cdiv(g.P, cols) + d / 2;
        return n > d ? n : d;
    };
    const int64_t nl = cdiv(rows, 256) * across(256), ns = cdiv(rows, 128) * across(128);
    // What either takes, in us, from the rates measured: HBM 5 MB, weights read again 12 MB, a stage of a small unit 0.85
    // us. Measured against each other (streaming, small tiles; us a call): K = 7168, N = 16384: T = 1 18, 29, 64 29, 30, 128 50, 30;
    // K = 14336, N = 4096, T = 128 30, 52; K = 2048, N = 16384, T = 128 31, 17; 64 experts, D = 7168, F = 2048, top 8:
    // T = 1 27, 37, 8 117, 118, 32 175, 183; D = 4096: T = 1 21, 23, 8 85, 74, 64 155, 120; back to D = 7168: 1 28, 25, 8 110, 81.
    const double mb = 1e-6 * (double)rows * (double)(g.kb() + g.sb());    // an expert's weights
    const double once = mb * (double)d, again = mb * (double)(across(16) - d);
    const double skinny = (once / 5 + again / 12) * (double)(steps + 4) / (double)steps + 3;
    const double small = (double)cdiv(ns, 2 * kCUs) * (0.85 * (double)steps + 4);
    if (skinny < (small > once / 5 ? small : once / 5) + once / 20) t = {kSkinny, 32, 16, 256, 0, 0, 0};
    // A round of large units takes half as long again as one of small ones, two to a compute unit (large, small; us a call): 64 experts,
    // D = 4096, F = 2048, top 8: T = 512 172, 167, 2048 266, 321; N = K = 4096: T = 2048 37, 32, 4096 50, 55. Where
    // that makes them equal, the gated projection takes large ones, the others small: T = 1024, 64 experts, top 8, D = 4096, F = 2048
    // 200, 213 and the projection back 156, 147.
    else if (3 * cdiv(nl, kCUs) < 2 * cdiv(ns, 2 * kCUs) + (g.op == kGlu ? 1 : 0)) t = {kLarge, 256, 256, 512, 0, 0, kCUs};
    else t = {kSmall, 128, 128, 256, 0, 0, 2 * kCUs};
    // Workgroups that take units in turn send off a unit's first loads before the last one's results are stored, and the stores
    // run beside its first products: T = 16384, K = 4096, N = 16384 643 against 661 us. The gated projection takes one unit each: in
    // this order its activation holds up the next unit, 714 against 702 us for 65536 pairs, D = 4096, F = 2048. (With the next unit's loads
    // beside the last products it took 655, but one run under a profiler's counters did not end, and no cause was found: not to be
    // taken up again without one. That loop had a second set of loads chosen by masks within the products, no meeting of the waves between
    // reduction and results, and scalar registers spilled to vector lanes, none of which the loop that is here has.)
    if (g.op == kGlu) t.places = 0;
    // A streaming workgroup can round its pairs' x rows itself, a launch and a workspace less, but each rounds them again. Two launches
    // against one, us a call: K = 7168, N = 16384: T = 1 17.5, 14.2, 7 17.1, 26.2; K = N = 4096: T = 4 16.7, 13.5, 12 16.2, 16.5;
    // K = 2048, N = 16384, T = 32 16.5, 24.2; T = 1, 64 experts, top 8: D = 7168, F = 2048 27.8, 29.0; D = 4096, F = 1024 22.1, 17.3.
    if (t.shape == kSkinny && x16) {
        const int64_t load = g.op == kProduct ? g.P : 2 * cdiv(g.P, g.E), pairs = load < 16 ? load : 16;
        t.rounds_x = g.P > 0 && pairs * g.K * cdiv(cdiv(rows, t.rows) * across(16), 2 * kCUs) <= 16384;
        const int64_t fit = kRoundedX / rounded_row(steps);      // more than `pairs`: 16384 values take 8704 bytes and half a stage each
        if (t.rounds_x && fit < t.cols) t.cols = (int)fit;
    }
    t.na = cdiv(rows, t.rows);
    // of the experts' buckets and that of the pairs without one
    t.nb = g.op == kProduct ? cdiv(g.P, t.cols) : g.P / t.cols + g.E + 1;
    if (t.nb > g.P) t.nb = g.P;
    return t;
}

inline bool valid(const Geometry& g)
{
    if (g.P < 0 || g.P > 0x7fffffff || g.X < 0) return false;
    if (g.E < 1 || g.E > kMaxE || g.share < 1 || g.share > kMaxTopK) return false;
    if (g.K < 1 || g.K > kMaxDim || g.R < 8 || g.R > kMaxDim || g.R % 8 != 0) return false;
    if (g.act != 0 && g.act != 1) return false;
    // x's codes are addressed in 31 bits
    if (g.X * g.kb() > 0x7fffffff) return false;
    if (mx::octet_blocks(g.X, g.K) < 0) return false;
    // the weighted sum: workgroups of 256 threads of eight results
    if (g.op == kDown && g.P * g.R / 2048 >= 0xffffff) return false;
    const Tiling t = make_tiling(g), r = make_tiling(g, true);
    return r.na * r.nb + 8 < (int64_t)1 << 23 && t.na * t.nb + 8 < (int64_t)1 << 23;     // workgroups of at most 512 threads within a grid's 2^32 - 1
}

// The projection back: whether the pairs' results, which the weighted sum reads, are kept in 16 bits, 11 of them
// significant, with a power of two for each 32 (mhc_experts.hip): where the caller allows it, for bf16, which has 8, in tiles.
inline bool parts_in_16_bits(const Geometry& g) { return g.op == kDown && g.short_terms && !g.f16 && make_tiling(g).shape != kSkinny; }
MHC_EXPERTS_HOST_DEVICE inline int64_t part_scales(int64_t R) { return (R + 31) / 32; }

struct Workspace {
    size_t off_codes = 0, off_scales = 0, off_part = 0, off_part_scales = 0, bytes = 0;
};
// quantise: x comes in 16 bits
inline Workspace make_workspace(const Geometry& g, bool quantise)
{
    Workspace w;
    size_t off = 0;
    quantise = quantise && !make_tiling(g, true).rounds_x;
    w.off_codes = off;
    if (quantise) off = align_up(off + (size_t)g.X * (size_t)g.kb(), 256);
    w.off_scales = off;
    if (quantise) off = align_up(off + (size_t)g.X * (size_t)g.sb(), 256);
    w.off_part = off;
    const bool in16 = parts_in_16_bits(g);
    if (g.op == kDown) off = align_up(off + (size_t)g.P * (size_t)g.R * (in16 ? 2 : 4), 256);
    w.off_part_scales = off;
    if (in16) off = align_up(off + (size_t)g.P * (size_t)part_scales(g.R), 256);
    w.bytes = off;
    return w;
}

// Unit t of an expert's na x nb units: the pairs of kGroup rows of units before the next rows', so that
// the units in flight on an XCD share a few operands of either kind in its L2.
constexpr uint32_t kGroup = 4;
MHC_EXPERTS_HOST_DEVICE inline void place(uint32_t t, uint32_t na, uint32_t nb, uint32_t* a, uint32_t* b)
{
    const uint32_t group = t / (kGroup * nb), r = t - group * kGroup * nb;
    const uint32_t rows = na - group * kGroup < kGroup ? na - group * kGroup : kGroup;
    *b = r / rows;
    *a = group * kGroup + (r - *b * rows);
}

// Bucket e's pairs [begin, end) by the plan's offsets, e = E those without an expert (and past that none). Whatever the
// offsets hold, pairs stay in [0, P).
MHC_EXPERTS_HOST_DEVICE inline void bucket_pairs(const int32_t* offsets, int E, int P, int e, int* begin, int* end)
{
    const int b = e <= E ? offsets[e] : P, n = e < E ? offsets[e + 1] : P;
    *begin = b < 0 ? 0 : (b > P ? P : b);
    *end = n < *begin ? *begin : (n > P ? P : n);
}
// Units of BC pairs that the buckets of a plan have at most. Sums of buckets' units stop there: offsets that are no plan's
// may name every pair in every bucket, and the sum of 1025 times P / BC units does not fit 32 bits. (64 buckets' does: valid() keeps
// P / BC under 2^23.)
MHC_EXPERTS_HOST_DEVICE inline int most_units(int64_t P, int BC, int E) { return (int)(P / BC) + E + 1; }
MHC_EXPERTS_HOST_DEVICE inline int units_sum(int at, int more, int most) { return at + more < most ? at + more : most; }
// Unit `unit` of before[E + 1] * na: its bucket e, its rows of units a and first pair; before[e]: the units along the pairs of the buckets before e.
MHC_EXPERTS_HOST_DEVICE inline void find_unit(const int* before, const int* begin, int E, uint32_t na, int BC, uint32_t unit, int* e, uint32_t* a,
                                              int64_t* first)
{
    const int q = (int)(unit / na);
    int at = 0, up = E + 1;                        // before[at] <= q < before[up]
    while (up - at > 1) {
        const int mid = (at + up) / 2;
        if (before[mid] <= q) at = mid;
        else up = mid;
    }
    uint32_t b;
    place(unit - (uint32_t)before[at] * na, na, (uint32_t)(before[at + 1] - before[at]), a, &b);
    *e = at;
    *first = begin[at] + (int64_t)b * BC;
}

struct Args {
    const uint16_t* x;            // [X, K] in 16 bits (a tiling that rounds it), or
    const uint8_t* x_codes;       // [X, kb]
    const uint8_t* x_scales;      // [X, sb]
    const uint8_t* w_codes[2];    // [E, R, kb] (the gated projection: gate and up)
    const uint8_t* w_scales[2];   // [E, R, sb]
    const int32_t* offsets;       // [E + 1], or NULL: one expert, pair i is row i
    const int32_t* pairs;         // [P]
    const float* weights;         // [P] (kDown)
    void* out;                    // [P, R] 16-bit (kDown: [P / k, R])
    void* part;                   // kDown: [P, R] fp32, or 16-bit with part_scales
    uint8_t* part_scales;         // [P, ceil(R / 32)]
    int64_t top_k;                // kDown
};

// Implemented in mhc_experts.hip. Returns 0 or the HIP error code.
int launch_products(const Geometry& g, const Tiling& t, const Args& a, void* stream);

}  // namespace experts
}  // namespace mhc
