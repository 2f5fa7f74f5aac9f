// Which kernel the launch plan takes: a line of op, T, k, E, D, F, x16 in (a plain product: K in the place of D, N in that of F),
// a line of validity, shape, units at most and workgroups that take units in turn (0: one for each) out.
#include <cstdio>

#include "mhc_experts_plan.h"

using namespace mhc::experts;

int main()
{
    long long T;
    int op, k, E, D, F, x16;
    while (scanf("%d %lld %d %d %d %d %d", &op, &T, &k, &E, &D, &F, &x16) == 7) {
        Geometry g;
        g.op = op;
        g.P = T * k;
        g.X = op == kDown ? g.P : T;
        g.E = E;
        g.share = op == kGlu ? k : 1;
        g.K = op == kDown ? F : D;
        g.R = op == kDown ? D : F;
        const Tiling t = make_tiling(g, x16 != 0);
        printf("%d %d %lld %lld\n", valid(g) ? 1 : 0, t.shape, (long long)(t.na * t.nb), (long long)t.places);
    }
    return 0;
}
