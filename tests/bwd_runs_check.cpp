// bwd_runs_check.cpp -- host-side check of which layout the backward's main pass takes for 16-bit x.
//
// Built with g++ by tests/test_bwd_runs_rule.py (no GPU, no HIP headers). Sizes at which one
// layout was measured to be the faster by 3 % and more. Prints "ok <cases>" or the first violation.
#include <cstdint>
#include <cstdio>

#include "mhc_bwd_plan.h"

using namespace mhc::bwd;

struct Case {
    int n, D, log2_values;
    bool gamma, xpost, f16, runs;
};

int main()
{
    const Case cases[] = {
        // few values, in rows of whole lines: the caches still join the pieces
        {4, 1024, 25, false, false, false, false}, {4, 2048, 25, false, false, true, false}, {4, 7168, 25, true, true, false, false},
        {6, 2048, 25, false, false, false, false}, {8, 1024, 25, true, true, true, false},
        // a last run that is mostly or partly empty
        {4, 136, 28, true, true, true, false}, {4, 160, 27, false, false, false, false}, {4, 192, 28, true, true, false, false},
        {4, 448, 28, true, false, true, false}, {6, 200, 28, true, true, false, false}, {8, 72, 28, false, false, false, false},
        {8, 520, 27, true, false, false, false},
        // large
        {4, 7168, 28, false, false, false, true}, {4, 7168, 28, true, true, true, true}, {4, 1024, 27, true, false, true, true},
        {4, 4104, 25, false, true, true, true}, {4, 232, 25, false, false, false, true}, {6, 4096, 28, true, true, false, true},
        {6, 4096, 28, false, false, true, true}, {8, 2048, 28, true, true, true, true}, {8, 1032, 26, false, true, true, true},
    };
    long long ok = 0;
    for (const Case& c : cases) {
        Geometry g;
        if (!make_geometry(c.n, c.D, &g, c.f16)) return std::printf("FAIL geometry n=%d D=%d\n", c.n, c.D), 1;
        const int64_t T = (((int64_t)1 << c.log2_values) + g.K - 1) / g.K;
        if (by_runs(g, T, c.gamma, c.xpost) != c.runs)
            return std::printf("FAIL n=%d D=%d 2^%d values gamma=%d xpost=%d f16=%d: expected %s\n", c.n, c.D, c.log2_values, c.gamma, c.xpost, c.f16,
                               c.runs ? "runs" : "d-blocks"), 1;
        ++ok;
    }
    // n = 8 without gradXPost has no kernel by runs, and no size may ask for one
    for (int D = 8; D <= 16384; D += 8)
        for (int f16 = 0; f16 < 2; ++f16) {
            Geometry g;
            if (!make_geometry(8, D, &g, f16) || by_runs(g, kMaxT, false, false) || by_runs(g, kMaxT, true, false))
                return std::printf("FAIL n=8 D=%d by runs\n", D), 1;
            ++ok;
        }
    std::printf("ok %lld\n", ok);
    return 0;
}
