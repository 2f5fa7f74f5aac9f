"""The pre-mapping's backward from 16-bit x where its main pass goes by runs, in every form that has such a kernel (n, gamma,
gradXPost, format): bit for bit what the same values give from their 8-bit checkpoint, whose kernels go by runs at every size and
are held against the oracle at small ones; and gradX, whose rows depend on their own token alone, bit for bit against calls on few
of the tokens, which go by d-blocks."""
import itertools
import sys

import pytest

from gpu_helpers import device

pytestmark = pytest.mark.gpu

# just past the sizes from which each form goes by runs (mhc_bwd_plan.h, by_runs), a last tile of few tokens
SHAPES = {4: [(24617, 1024), (6149, 4104)], 6: [(15433, 1088)], 8: [(11579, 1088)]}
CASES = [(T, n, D, *c) for n, shapes in SHAPES.items() for T, D in shapes for c in itertools.product((False, True), repeat=3) if n != 8 or c[1]]
CASES += [(8401, 6, 1000, False, True, True), (6301, 8, 1000, False, True, True)]      # a last block of 8 positions


@pytest.mark.parametrize("T,n,D,gamma,post,f16", CASES)
def test_runs_give_the_bits_of_the_other_layouts(T, n, D, gamma, post, f16):
    import mhc_hyper_connection_amd as mhc
    import torch
    dev, dt, M = device(), torch.float16 if f16 else torch.bfloat16, n * n + 2 * n
    print(f"[case] backward layouts T={T} n={n} D={D} gamma={gamma} post={post} f16={f16}", file=sys.stderr, flush=True)
    g = torch.Generator(device=dev).manual_seed(T)
    f32 = lambda *s: torch.randn(*s, generator=g, device=dev)
    ck = mhc.mhc_checkpoint(f32(T, n, D).to(dt))
    x = mhc.mhc_checkpoint_restore(ck)
    gate = torch.rand((T, 2 * n), generator=g, device=dev)
    per_token = [f32(T, D).to(dt), f32(T, n), f32(T, n, n), f32(T).abs() + 0.5, f32(T, M), gate[:, :n].contiguous(), gate[:, n:].contiguous()]
    phi, alpha, gam = f32(M, n * D) * (n * D) ** -0.5, f32(3), f32(n, D) if gamma else None
    xp = f32(T, n, D).to(dt) if post else None

    def run(x, s):
        t = [v[s] for v in per_token]
        return mhc.mhc_pre_backward(x, phi, alpha, *t, gam, None if xp is None else xp[s])

    whole = run(x, slice(0, T))
    kept = run(ck, slice(0, T))
    for k in whole:
        assert torch.isfinite(whole[k]).all(), k
        assert torch.equal(whole[k].view(torch.uint8), kept[k].view(torch.uint8)), k
    for lo, hi in ((0, 1), (0, 130), (T // 2, T // 2 + 65), (T - 67, T)):
        assert torch.equal(whole["grad_x"][lo:hi].view(torch.int16), run(x[lo:hi], slice(lo, hi))["grad_x"].view(torch.int16)), (lo, hi)
