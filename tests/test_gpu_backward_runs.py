"""GPU parity of the MhcPre backward where x is large (2^25 values and more): the main pass then
takes runs of one stream's positions. Every form of the kernel (n, gamma, gradXPost, format) at sizes
whose last run, last block of 32 positions and last tile of tokens are partial, against the fp64
oracle, with test_gpu_backward's acceptance rule; and gradX, whose rows depend on their own token
alone, bit for bit against calls on few of the tokens, which take the other layout.
"""
import itertools

import pytest

import synth
from gpu_helpers import device, to_dev
from test_gpu_backward import compare, gpu_backward, run_oracle

pytestmark = pytest.mark.gpu

SHAPES = [(2045, 4, 4104), (2721, 6, 2056), (4065, 8, 1032)]
CASES = [(*s, *c) for s in SHAPES for c in itertools.product((False, True), repeat=3)]
CASES += [(61700, 4, 136, True, True, False), (61700, 4, 136, False, False, True)]


@pytest.mark.parametrize("T,n,D,gamma,post,f16", CASES)
def test_large_x_by_runs(T, n, D, gamma, post, f16):
    assert T * n * D >= 1 << 25
    bi = synth.backward_inputs(T, n, D, gamma=gamma, x_post=post, seed=T + D + n, x_f16=f16)
    compare(gpu_backward(bi), run_oracle(bi), bi)


@pytest.mark.parametrize("T,n,D", SHAPES)
@pytest.mark.parametrize("f16", [False, True])
def test_grad_x_of_few_tokens_is_the_same(T, n, D, f16):
    import mhc_hyper_connection_amd as mhc
    import torch
    bi = synth.backward_inputs(T, n, D, gamma=True, x_post=True, seed=n, x_f16=f16)
    dev = device()
    x, phi, alpha, gi, gp, gr, ir, hm, hp, ho, gamma, xp = [
        to_dev(a, dev, f16) for a in (bi.x, bi.phi, bi.alpha, bi.grad_h_in, bi.grad_h_post, bi.grad_h_res, bi.inv_rms,
                                      bi.h_mix, bi.h_pre, bi.h_post, bi.gamma, bi.grad_x_post)]
    def grad_x(lo, hi):
        return mhc.mhc_pre_backward(x[lo:hi], phi, alpha, gi[lo:hi], gp[lo:hi], gr[lo:hi], ir[lo:hi], hm[lo:hi], hp[lo:hi],
                                    ho[lo:hi], gamma, xp[lo:hi], hc_eps=bi.hc_eps)["grad_x"].clone()
    whole = grad_x(0, T)
    for lo, hi in ((0, 1), (0, 130), (T // 2, T // 2 + 65), (T - 67, T)):
        assert torch.equal(whole[lo:hi].view(torch.int16), grad_x(lo, hi).view(torch.int16)), (lo, hi)
