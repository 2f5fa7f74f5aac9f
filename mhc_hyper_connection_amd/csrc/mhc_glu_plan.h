// mhc_glu_plan.h -- geometry, launch shapes and workspace layout of the gated projection
// h = act(x Wg^T) (.) (x Wu^T) and its backward.
//
// Host-side and plain C++ (no HIP headers), like mhc_plan.h.
#pragma once

#include <cstddef>
#include <cstdint>

#ifdef __HIP__
#define MHC_GLU_HOST_DEVICE __host__ __device__
#else
#define MHC_GLU_HOST_DEVICE
#endif

namespace mhc {
namespace glu {

constexpr int kMaxD = 16384;
constexpr int kMaxF = 65536;
constexpr int kBK = 64;              // reduction positions per LDS stage
constexpr int kCUs = 256;

struct Geometry {
    int64_t T = 0;
    int D = 0, F = 0;
    int act = 0;       // 0 SiLU, 1 GELU (tanh form)
    int f16 = 0;
    // Few tokens: the kernel that streams the weights past all of them. Up to 32 tokens it is
    // the faster at every size measured (D = 7168, F = 14336: 71 us against the tiles' 78 for
    // one token, 74 against 85 for 16, 88 against 89 for 32; D = F = 4096: 15 against 32
    // for 16); up to 64 while the tiles would leave half the compute units empty (64 tokens:
    // D = F = 4096 18 us against 33, F = 14336 110 against 94).
    bool skinny() const { return T <= 32 || (T <= 64 && F <= 8192); }
};

inline bool make_geometry(int64_t T, int D, int F, int act, int f16, Geometry* g)
{
    if (T < 0 || T > (int64_t)1 << 31) return false;
    if (D < 8 || D % 8 != 0 || D > kMaxD) return false;
    if (F < 8 || F % 8 != 0 || F > kMaxF) return false;
    if (act != 0 && act != 1) return false;
    g->T = T;
    g->D = D;
    g->F = F;
    g->act = act;
    g->f16 = f16;
    // tiles of 128 tokens x 64 f: workgroups within a grid's 2^32 - 1 threads
    return ((T + 127) / 128) * ((F + 63) / 64) < (int64_t)1 << 23;
}

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// A tiled product of `rows` x `cols` results over `steps` stages of kBK, in 256 x 256 tiles
// (one workgroup of 8 waves per compute unit) or 128 x 128 tiles (4 waves, two workgroups
// per compute unit). Tiles run in rounds of one for each place on the chip; where the last
// round would leave places empty and the product may be split (its results are plain sums),
// each of its tiles is cut along the reduction into as many parts as fill it, whose fp32
// results a second kernel joins.
struct Tiling {
    bool large = false;
    int64_t na = 0, nb = 0;   // tiles along rows and columns
    int64_t whole = 0;        // tiles not cut: the first of the tile order
    int split = 1;            // parts of each of the others
    int64_t steps = 0;        // stages in all
    int64_t per = 0;          // stages of a part
    int64_t rest() const { return na * nb - whole; }
    // workgroups: both runs padded to whole turns of the 8 XCDs
    int64_t blocks() const { return (whole + 7) / 8 * 8 + (rest() * split + 7) / 8 * 8; }
    size_t part_bytes() const { return (size_t)(rest() * split) * (large ? 256 * 256 : 128 * 128) * 4; }
};
// groups: independent products of this size in one launch (2 for the two weights' gradients)
inline Tiling make_tiling(int64_t rows, int64_t cols, int64_t steps, int groups, bool may_split)
{
    Tiling t;
    t.steps = steps;
    // Rounds of large tiles against rounds of two small ones per compute unit, which take
    // 2/3 of a large one's time; a product that may be split fills its last round, and is
    // worth large tiles once every compute unit has 4 stages of one.
    const int64_t nl = cdiv(rows, 256) * cdiv(cols, 256) * groups, ns = cdiv(rows, 128) * cdiv(cols, 128) * groups;
    t.large = may_split ? nl * steps >= 4 * kCUs : 3 * cdiv(nl, kCUs) <= 2 * cdiv(ns, 2 * kCUs);
    const int64_t tile = t.large ? 256 : 128, places = t.large ? kCUs : 2 * kCUs;
    t.na = cdiv(rows, tile);
    t.nb = cdiv(cols, tile) * groups;
    const int64_t tiles = t.na * t.nb;
    t.whole = tiles;
    t.per = steps;
    if (!may_split || tiles == 0 || steps == 0) return t;
    const int64_t rest = tiles % places;
    int64_t s = rest ? places / rest : 1;
    if (s > steps / 4) s = steps / 4;     // parts of at least 4 stages
    if (s < 2) return t;
    t.per = cdiv(steps, s);
    t.split = (int)cdiv(steps, t.per);
    t.whole = tiles - rest;
    return t;
}

// Workgroup -> tile and part. Workgroups b, b + 8, .. run on one XCD; each XCD takes a
// contiguous run of the tile order, which walks the columns of kGroup rows of tiles before the
// next rows: the tiles in flight on an XCD then share kGroup row operands and a few column
// operands in its L2 (4 against 2, 8 and 16: within 2 % of the best for every product). The
// cut tiles follow, the same part of neighbouring tiles side by side. False for the padding
// of an XCD's run.
constexpr uint32_t kGroup = 4;
struct Unit {
    uint32_t a, b, tile;   // tile row, tile column, place in the order
    int part;              // -1: the whole tile
};
MHC_GLU_HOST_DEVICE inline void place(uint32_t t, uint32_t na, uint32_t nb, Unit* u)
{
    const uint32_t group = t / (kGroup * nb), r = t - group * kGroup * nb;
    const uint32_t rows = na - group * kGroup < kGroup ? na - group * kGroup : kGroup;
    u->tile = t;
    u->b = r / rows;
    u->a = group * kGroup + (r - u->b * rows);
}
MHC_GLU_HOST_DEVICE inline bool unit_of(uint32_t block, uint32_t na, uint32_t nb, uint32_t whole, uint32_t split, Unit* u)
{
    const uint32_t first = (whole + 7) / 8;          // of the whole tiles, on each XCD
    const uint32_t xcd = block % 8, i = block / 8;
    if (i < first) {
        const uint32_t t = xcd * first + i;
        if (t >= whole) return false;
        u->part = -1;
        place(t, na, nb, u);
        return true;
    }
    const uint32_t rest = na * nb - whole, units = rest * split, per = (units + 7) / 8;
    const uint32_t v = xcd * per + (i - first);
    if (i - first >= per || v >= units) return false;
    u->part = (int)(v / rest);
    place(whole + v % rest, na, nb, u);
    return true;
}

struct BackwardPlan {
    Tiling act, dx, dw;       // recomputed projections; x's gradient; the weights' gradients
    size_t off_dgu = 0, off_x = 0, off_part = 0, ws_bytes = 0;
};

inline Tiling forward_tiling(const Geometry& g) { return make_tiling(2 * (int64_t)g.F, g.T, cdiv(g.D, kBK), 1, false); }

inline BackwardPlan make_backward_plan(const Geometry& g, bool checkpoint)
{
    BackwardPlan p;
    p.act = forward_tiling(g);
    p.dx = make_tiling(g.D, g.T, 2 * cdiv(g.F, kBK), 1, true);
    p.dw = make_tiling(g.D, g.F, cdiv(g.T, kBK), 2, true);
    size_t off = 0;
    p.off_dgu = off;
    off = align_up(off + (size_t)g.T * 2 * (size_t)g.F * 2, 256);
    p.off_x = off;
    if (checkpoint) off = align_up(off + (size_t)g.T * (size_t)g.D * 2, 256);
    p.off_part = off;
    const size_t px = p.dx.part_bytes(), pw = p.dw.part_bytes(), part = px > pw ? px : pw;
    off = align_up(off + part, 256);
    p.ws_bytes = off;
    return p;
}

struct Args {
    const uint16_t* x;        // [T, D]
    const uint16_t* w_gate;   // [F, D]
    const uint16_t* w_up;     // [F, D]
    uint16_t* h;              // [T, F] (the backward: may be NULL)
    // backward
    const uint16_t* grad_h;   // [T, F]
    uint16_t* grad_x;         // [T, D]
    uint16_t* grad_w_gate;    // [F, D]
    uint16_t* grad_w_up;      // [F, D]
    uint16_t* dgu;            // [T, 2F] gradients of the two projections' results
    float* part;
};

// Implemented in mhc_glu.hip. Each returns 0 or the HIP error code.
int launch_glu(const Geometry& g, const Args& a, void* stream);
int launch_glu_backward(const Geometry& g, const BackwardPlan& p, const Args& a, void* stream);

}  // namespace glu
}  // namespace mhc
