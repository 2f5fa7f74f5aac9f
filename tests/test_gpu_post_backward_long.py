"""hc_post's backward on the GPU over more tokens than one launch takes (64 threads a token, 2^32 - 1 threads a grid): the
tokens on both sides of the launches' border, the first and the last give what they give by themselves."""
import sys

import pytest

from gpu_helpers import device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kept", [False, True])
def test_more_tokens_than_a_launch_takes(kept):
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    n, D, border = 4, 8, 4 * 0xFFFFFF
    T = border + 70
    print(f"[case] post_backward T={T} n={n} D={D} kept={kept}", file=sys.stderr, flush=True)
    bf = dict(dtype=torch.bfloat16, device=dev)
    t = dict(grad_out=torch.zeros((T, n, D), **bf), x=torch.zeros((T, D), **bf), residual=torch.zeros((T, n, D), **bf),
             post=torch.zeros((T, n), device=dev), comb=torch.zeros((T, n, n), device=dev))
    spans = [slice(0, 9), slice(border - 66, border + 66), slice(T - 3, T)]
    g = torch.Generator(device=dev).manual_seed(4)
    for s in spans[:2] + [slice(border + 66, T)]:
        for v in t.values():
            v[s] = torch.randn(v[s].shape, generator=g, device=dev).to(v.dtype)

    def run(s):
        a = {k: v[s] for k, v in t.items()}
        keep = mhc.mhc_checkpoint if kept else (lambda v: v)
        return mhc.mhc_post_backward(a["grad_out"], keep(a["x"]), keep(a["residual"]), a["post"], a["comb"])

    whole = run(slice(0, T))
    torch.cuda.synchronize()
    # 512 tokens and more of D = 8 take one wave a token, as the whole does: each span within 600
    for s in spans:
        lo = max(0, min(s.start, T - 600))
        small = run(slice(lo, lo + 600))
        for k in whole:
            assert torch.equal(whole[k][s], small[k][s.start - lo:s.stop - lo]), (k, s)
    for k in whole:                                   # and the zeros between stay zeros
        assert not whole[k][9:border - 66].any(), k
