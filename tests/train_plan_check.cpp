// train_plan_check.cpp -- host-side bounds checks of the training operators' launch plans.
//
// Built with g++ by tests/test_train_plan.py (no GPU, no HIP headers). For a sweep of sizes it
// replays, with the helpers the kernels use (mhc_glu_plan.h, mhc_bwd_plan.h,
// mhc_train_plan.h), which tile, part, run and stream each workgroup takes, the stages of the parts, the
// 32-bit offsets of the tiles' loads and the workspace sections. Prints "ok <cases>" or the first violation.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "mhc_bwd_plan.h"
#include "mhc_glu_plan.h"
#include "mhc_train_plan.h"

using namespace mhc;

static int fail(const char* what, long long T, int D, int F, long long a, long long b)
{
    std::printf("FAIL %s T=%lld D=%d F=%d (%lld vs %lld)\n", what, T, D, F, a, b);
    return 1;
}

static int check_tiling(const glu::Tiling& t, long long T, int D, int F, bool may_split)
{
    const long long tiles = t.na * t.nb, blocks = t.blocks(), threads = blocks * (t.large ? 512 : 256);
    if (threads >= 1LL << 32) return fail("grid", T, D, F, threads, 0);
    if (t.whole < 0 || t.whole > tiles || (!may_split && t.whole != tiles)) return fail("whole tiles", T, D, F, t.whole, tiles);
    if (tiles == 0) return 0;
    if (t.split < 1 || (t.rest() > 0 && t.split < 2)) return fail("split", T, D, F, t.split, t.rest());
    if (t.rest() > 0 && ((t.split - 1) * t.per >= t.steps || t.split * t.per < t.steps)) return fail("parts", T, D, F, t.per, t.steps);
    if (t.rest() * t.split > (t.large ? 1 : 2) * glu::kCUs) return fail("places", T, D, F, t.rest() * t.split, 0);
    if (tiles > 2000000) return 0;
    std::vector<char> whole((size_t)tiles, 0), parts((size_t)(t.rest() * t.split), 0);
    std::vector<char> at((size_t)tiles, 0);
    for (long long b = 0; b < blocks; ++b) {
        glu::Unit u;
        if (!glu::unit_of((uint32_t)b, (uint32_t)t.na, (uint32_t)t.nb, (uint32_t)t.whole, (uint32_t)t.split, &u)) continue;
        if (u.a >= t.na || u.b >= t.nb || u.tile >= tiles) return fail("tile range", T, D, F, u.a, u.b);
        char& seen = u.part < 0 ? whole[u.tile] : parts[(size_t)((u.tile - t.whole) * t.split + u.part)];
        if ((u.part < 0) != (u.tile < t.whole) || u.part >= t.split || seen) return fail("unit twice", T, D, F, u.tile, u.part);
        seen = 1;
        if (u.part <= 0) {
            if (at[(size_t)u.a * t.nb + u.b]) return fail("tile twice", T, D, F, u.a, u.b);
            at[(size_t)u.a * t.nb + u.b] = 1;
        }
    }
    for (long long i = 0; i < tiles; ++i)
        if (!at[(size_t)i] || (i < t.whole && !whole[(size_t)i])) return fail("tile missing", T, D, F, i, tiles);
    for (char c : parts)
        if (!c) return fail("part missing", T, D, F, 0, 0);
    return 0;
}

static int check_glu(long long T, int D, int F)
{
    glu::Geometry g;
    if (!glu::make_geometry(T, D, F, 0, 0, &g)) return fail("geometry", T, D, F, 0, 0);
    for (int ck = 0; ck < 2; ++ck) {
        const glu::BackwardPlan p = glu::make_backward_plan(g, ck == 1);
        if (check_tiling(p.act, T, D, F, false) || check_tiling(p.dx, T, D, F, true) || check_tiling(p.dw, T, D, F, true)) return 1;
        const size_t off[] = {p.off_dgu, p.off_x, p.off_part, p.ws_bytes};
        const size_t need[] = {(size_t)T * 2 * F * 2, ck ? (size_t)T * D * 2 : 0, p.dx.part_bytes() > p.dw.part_bytes() ? p.dx.part_bytes() : p.dw.part_bytes()};
        for (int s = 0; s < 3; ++s)
            if (off[s] % 256 || off[s] + need[s] > off[s + 1]) return fail("section", T, D, F, s, (long long)need[s]);
        if (T > 0 && (p.dx.steps * glu::kBK < 2LL * F || p.dw.steps * glu::kBK < T || p.act.steps * glu::kBK < D)) return fail("stages", T, D, F, 0, 0);
    }
    // byte offsets of a tile's loads: a tile's rows contiguous along the reduction, and a stage's
    // rows across it, up to the padding of the last tile
    const long long far[] = {256LL * D * 2, 256LL * 2 * F * 2 + 2LL * (2 * F + 2 * glu::kBK), (glu::kBK - 1) * 2LL * D + 2LL * (D + 512),
                             (glu::kBK - 1) * 4LL * F + 2LL * (2 * F + 512), 64LL * D * 2};
    for (long long v : far)
        if (v >= 1LL << 31) return fail("offset", T, D, F, v, 0);
    return 0;
}

static int check_runs(int n, int D, long long T)
{
    bwd::Geometry g;
    if (!bwd::make_geometry(n, D, &g)) return fail("backward geometry", T, D, n, 0, 0);
    const bwd::Plan p = bwd::make_plan(g, T);
    const int runs = (g.nblk + g.SGN - 1) / g.SGN;
    const long long tasks = bwd::run_tasks_for(p.G, g.nblk, g.SGN, n), blocks = bwd::run_blocks_for(tasks, n);
    if (blocks < tasks || blocks % (8 * n) || blocks * 256 >= 1LL << 32) return fail("run blocks", T, D, n, blocks, tasks);
    std::vector<long long> at((size_t)tasks, -1);
    for (long long b = 0; b < blocks; ++b) {
        int64_t gr;
        int run, st;
        if (!bwd::run_task(b, runs, n, tasks, &gr, &run, &st)) continue;
        if (gr < 0 || gr >= p.G || run < 0 || run >= runs || st < 0 || st >= n) return fail("run range", T, D, n, gr, run);
        const size_t id = ((size_t)gr * runs + run) * n + st;
        if (at[id] >= 0) return fail("run twice", T, D, n, b, (long long)id);
        at[id] = b;
        if (bwd::pack_at(run * g.SGN, st, n, g.KS) + bwd::pack_units_per_stream(g.KS) > (int64_t)(g.pack_bytes / 16)) return fail("pack", T, D, n, run, st);
    }
    for (size_t id = 0; id < at.size(); ++id) {
        if (at[id] < 0) return fail("run missing", T, D, n, (long long)id, 0);
        if (id % n && at[id] - at[id - 1] != 8) return fail("a run's streams not on one XCD", T, D, n, at[id], at[id - 1]);
    }
    return 0;
}

int main()
{
    long long cases = 0;
    const int Ds[] = {8, 16, 24, 40, 256, 264, 1000, 2048, 4096, 7168, 16384}, Fs[] = {8, 24, 64, 200, 520, 4104, 8192, 14336, 65536};
    const long long Ts[] = {0, 1, 16, 17, 64, 65, 127, 129, 257, 1003, 4096, 16384, 100003};
    for (int D : Ds)
        for (int F : Fs)
            for (long long T : Ts) {
                if (check_glu(T, D, F)) return 1;
                ++cases;
            }
    for (int n : {4, 6, 8})
        for (int D : Ds)
            for (long long T : {1LL, 63LL, 65LL, 4096LL, 16384LL, 100003LL}) {
                if (check_runs(n, D, T)) return 1;
                ++cases;
            }
    for (int D : Ds)   // rows x padded octets: the last grid that is taken and the first that is not
        for (long long rows : {1LL, 255LL, 0xffffffLL * 256 / ckpt_octets(D)}) {
            const long long b = octet_blocks(rows, D);
            if (b < 1 || b * 256 < rows * ckpt_octets(D) || b * 256 >= 1LL << 32) return fail("octet blocks", rows, D, 0, b, 0);
            if (octet_blocks(0xffffffLL * 256 / ckpt_octets(D) + 1, D) != -1) return fail("octet blocks refused", rows, D, 0, 0, 0);
            ++cases;
        }
    std::printf("ok %lld\n", cases);
    return 0;
}
