// post_bwd_plan_check.cpp -- host-side check of the launches of hc_post's backward.
//
// Built with g++ by tests/test_post_bwd_plan.py (no GPU, no HIP headers). For every size that
// the entry point takes, at its largest T and around a launch's most tokens, with the helpers
// that the launcher uses (mhc_train_plan.h): each grid's threads, the tokens that the launches
// cover, and where each launch's pointers stand. Prints "ok <cases>" or the first violation.
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "mhc_train_plan.h"

using namespace mhc;

template <class P>
static long long at(P* p) { return (long long)reinterpret_cast<uintptr_t>(p); }

int main()
{
    long long cases = 0;
    for (int n : {4, 6, 8})
        for (int D = 8; D <= 16384; D += 8) {
            const int64_t last = (int64_t)0xffffff * 256 / ckpt_octets(D);   // the most that octet_blocks takes
            for (int64_t T : {(int64_t)1, (int64_t)511, (int64_t)512, (int64_t)0xffffff, (int64_t)0xffffff + 1, (int64_t)4 * 0xffffff,
                              (int64_t)4 * 0xffffff + 1, (int64_t)9 * 0xffffff, last}) {
                if (T > last) continue;
                if (octet_blocks(T, D) < 1) return std::printf("FAIL refused T=%lld D=%d\n", (long long)T, D), 1;
                const int W = post_bwd_waves(T, n, D);
                const int64_t most = post_bwd_launch_tokens(W);
                PostBwdArgs a = {};
                int64_t done = 0;
                for (int64_t left = T; left > 0; left -= most) {
                    const int64_t Tc = left < most ? left : most, blocks = post_bwd_blocks(Tc, W);
                    if (blocks < 1 || blocks * 256 > 0xffffffffLL) return std::printf("FAIL grid T=%lld n=%d D=%d: %lld\n", (long long)T, n, D, (long long)blocks), 1;
                    if (blocks * (W == 1 ? 4 : 1) < Tc) return std::printf("FAIL tokens T=%lld n=%d D=%d\n", (long long)T, n, D), 1;
                    // x as codes, residual as codes: pointers from zero are the offsets in bytes
                    const long long want[] = {done * n * D * 2, done * D, done * ckpt_blocks(D), done * n * D, done * n * ckpt_blocks(D), done * n * 4,
                                              done * n * n * 4, done * D * 2, done * n * D * 2, done * n * 4, done * n * n * 4};
                    const long long got[] = {at(a.grad_out), at(a.x_codes), at(a.x_scales), at(a.r_codes), at(a.r_scales), at(a.post), at(a.comb),
                                             at(a.grad_x), at(a.grad_residual), at(a.grad_post), at(a.grad_comb)};
                    for (int k = 0; k < 11; ++k)
                        if (got[k] != want[k]) return std::printf("FAIL pointer %d T=%lld n=%d D=%d\n", k, (long long)T, n, D), 1;
                    done += Tc;
                    if (left > most) a = post_bwd_after(a, Tc, n, D);
                }
                if (done != T) return std::printf("FAIL covered T=%lld n=%d D=%d: %lld\n", (long long)T, n, D, (long long)done), 1;
                ++cases;
            }
        }
    // 16-bit activations: their pointers move, the absent checkpoints' stay NULL
    uint16_t x[3 * 8], r[3 * 4 * 8];
    PostBwdArgs a = {};
    a.x = x;
    a.residual = r;
    a = post_bwd_after(a, 2, 4, 8);
    if (a.x != x + 16 || a.residual != r + 64 || a.x_codes || a.x_scales || a.r_codes || a.r_scales) return std::printf("FAIL 16-bit pointers\n"), 1;
    std::printf("ok %lld\n", cases);
    return 0;
}
