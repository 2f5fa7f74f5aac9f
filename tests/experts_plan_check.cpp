// Replays the launch plans of the routing plan and of the products with 4-bit weights on the host: every result is of
// exactly one unit, no unit passes its expert's pairs or the weights' rows, and the grid holds every unit whatever
// the experts' loads are.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "mhc_experts_plan.h"
#include "mhc_route_plan.h"

using namespace mhc;

static uint64_t state = 88172645463325252ull;
static uint32_t rnd(uint32_t n)
{
    state ^= state << 13;
    state ^= state >> 7;
    state ^= state << 17;
    return (uint32_t)(state % n);
}
static int fail(const char* what, long long a, long long b)
{
    printf("FAIL %s %lld %lld\n", what, a, b);
    return 1;
}

static int check_units(const experts::Geometry& g, const std::vector<int64_t>& load, bool x16)
{
    const experts::Tiling t = experts::make_tiling(g, x16);
    if (t.cols < 1 || (t.rounds_x && (!x16 || t.shape != experts::kSkinny || t.cols > 16 ||
                                      t.cols * experts::rounded_row(experts::cdiv(g.kb(), 128)) > experts::kRoundedX)))
        return fail("rounded rows", t.cols, g.K);
    const int64_t rows = g.op == experts::kGlu ? 2 * (int64_t)g.R : g.R;
    if (t.na * t.rows < rows || (t.na - 1) * t.rows >= rows) return fail("rows", t.na, rows);
    // what the kernel counts: the buckets' units, expert by expert
    std::vector<int64_t> nb(load.size()), before(load.size() + 1, 0);
    for (size_t e = 0; e < load.size(); ++e) {
        nb[e] = (load[e] + t.cols - 1) / t.cols;
        before[e + 1] = before[e] + nb[e];
    }
    const int64_t total = before.back(), units = total * t.na, grid = t.grid(), per = (units + 7) / 8;
    if (total > t.nb) return fail("units past the grid's", total, t.nb);
    if (grid % 8 || grid > 8 * experts::cdiv(t.na * t.nb, 8)) return fail("grid", grid, t.nb);
    if (!t.places && (per - 1) * 8 + 7 >= grid && units > 0) return fail("grid", per, grid);
    std::vector<char> seen((size_t)units, 0);
    for (int64_t b = 0; b < grid; ++b) {
      int64_t taken = 0;
      for (int64_t i = b / 8; i < per; i += t.places ? grid / 8 : per) {
        if (++taken > 64) return fail("a workgroup's units", grid, per);
        const int64_t u = (b % 8) * per + i;
        if (u >= units) break;
        const int64_t q = u / t.na;
        size_t e = 0;
        while (q >= before[e + 1]) ++e;
        uint32_t a, c;
        experts::place((uint32_t)(u - before[e] * t.na), (uint32_t)t.na, (uint32_t)nb[e], &a, &c);
        if (a >= t.na || c >= nb[e]) return fail("place", a, c);
        char& s = seen[(size_t)(before[e] * t.na + (int64_t)c * t.na + a)];
        if (s) return fail("twice", (long long)e, u);
        s = 1;
      }
    }
    for (char s : seen)
        if (!s) return fail("never", units, total);
    return 0;
}

int main()
{
    long long n = 0, rounds = 0;
    for (int it = 0; it < 4000; ++it) {
        experts::Geometry g;
        g.op = (int)rnd(3);
        g.E = g.op == experts::kProduct ? 1 : 1 + (int)rnd(it % 3 ? 20 : 300);
        g.K = 1 + (int)rnd(it % 4 ? 300 : 20000);
        g.R = 8 * (1 + (int)rnd(it % 5 ? 60 : 600));
        std::vector<int64_t> load;
        const uint32_t most = 1 + rnd(it % 7 ? 80 : 2000);
        for (int e = 0; e < g.E; ++e) load.push_back(rnd(3) ? rnd(most) : 0);
        if (g.op != experts::kProduct) load.push_back(rnd(2) ? rnd(most) : 0);    // pairs without an expert
        for (int64_t l : load) g.P += l;
        g.X = g.P;
        if (g.P == 0) continue;
        if (!experts::valid(g)) return fail("valid", g.P, g.R);
        if (check_units(g, load, false) || check_units(g, load, true)) return 1;
        // the same pairs all with one expert
        std::vector<int64_t> one(load.size(), 0);
        one[rnd((uint32_t)load.size())] = g.P;
        if (check_units(g, one, false) || check_units(g, one, true)) return 1;
        for (int q = 0; q < 2; ++q) {
            const experts::Workspace w = experts::make_workspace(g, q == 1);
            const bool quantised = q == 1 && !experts::make_tiling(g, true).rounds_x;
            rounds += q == 1 && !quantised;
            const bool in16 = experts::parts_in_16_bits(g);
            const int64_t need = (quantised ? g.X * (g.kb() + g.sb()) : 0) + (g.op != experts::kDown ? 0 : in16 ? g.P * g.R * 2 + g.P * experts::part_scales(g.R) : g.P * g.R * 4);
            if (in16 && (w.off_part_scales % 256 || (int64_t)(w.off_part_scales - w.off_part) < g.P * g.R * 2)) return fail("parts", g.P, g.R);
            if ((int64_t)w.bytes < need || w.off_codes % 256 || w.off_scales % 256 || w.off_part % 256) return fail("workspace", (long long)w.bytes, need);
            if (quantised && (int64_t)(w.off_scales - w.off_codes) < g.X * g.kb()) return fail("codes", (long long)w.off_scales, g.X);
            if (quantised && g.op == experts::kDown && (int64_t)(w.off_part - w.off_scales) < g.X * g.sb()) return fail("scales", (long long)w.off_part, g.X);
        }
        ++n;
    }
    if (rounds < 100) return fail("few that round x", rounds, n);
    // the routing plan's chunks cover the pairs once
    for (int it = 0; it < 20000; ++it) {
        route::Plan p;
        const int64_t pairs = it < 9000 ? it : (int64_t)rnd(0x7fffffff);
        if (!route::make_plan(pairs, 1 + (int)rnd(1024), &p)) return fail("plan", pairs, 0);
        if (p.chunks < 1 || p.chunks > route::kPlanChunks || p.chunks * p.chunk < pairs) return fail("chunks", p.chunks, p.chunk);
        if (p.chunks > 1 && ((p.chunks - 1) * p.chunk >= pairs || p.ws_bytes != (size_t)p.chunks * (size_t)(p.E + 1) * 4)) return fail("last chunk", pairs, p.chunk);
        ++n;
    }
    printf("ok %lld\n", n);
    return 0;
}
