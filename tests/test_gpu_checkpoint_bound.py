"""The error bound that the 8-bit checkpoint promises, down to the least values of both formats, and scale bytes at any
address: exact arithmetic, so nothing here has a tolerance beside the bound itself."""
import sys

import numpy as np
import pytest

import synth
from gpu_helpers import device, to_dev
from train_helpers import BLOCK, to_16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("f16", [False, True])
def test_error_bound_at_every_size_of_a_block(f16):
    # a block for each power of two that the format has, its other values anywhere up to it
    import mhc_hyper_connection_amd as mhc
    rng = np.random.default_rng(6)
    top = np.arange(-24, 16) if f16 else np.arange(-133, 128)
    a = np.exp2(top.astype(np.float64))[:, None] * np.concatenate([np.ones((len(top), 1)), rng.uniform(-2, 2, (len(top), BLOCK - 1))], 1)
    a = np.clip(a, -65504.0, 65504.0) if f16 else np.clip(a, -3.3895313892515355e38, 3.3895313892515355e38)
    x = to_16(a, f16)
    v = x.double().numpy()
    print(f"[case] checkpoint bound f16={f16}", file=sys.stderr, flush=True)
    back = mhc.mhc_checkpoint_restore(mhc.mhc_checkpoint(x.to(device()))).double().cpu().numpy()
    off, biggest = np.abs(back - v), np.abs(v).max(1, keepdims=True)
    assert (off <= np.maximum(biggest / 128, 2.0 ** -127)).all()
    if f16:
        assert (off <= biggest / 128).all()
    else:   # a block of 2^-127 alone is half its step and comes back as 0: the bound's second part is reached
        one = to_16(np.full((1, 8), 2.0 ** -127), False)
        assert not mhc.mhc_checkpoint_restore(mhc.mhc_checkpoint(one.to(device()))).any()


@pytest.mark.parametrize("n,D", [(4, 264), (6, 1000), (8, 96)])
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_scale_bytes_at_any_address(n, D, shift):
    # scales have no alignment of their own: a checkpoint whose bytes start anywhere gives the same bits
    import mhc_hyper_connection_amd as mhc
    import torch
    T, dev = 133, device()
    print(f"[case] checkpoint scales n={n} D={D} shift={shift}", file=sys.stderr, flush=True)
    bi = synth.backward_inputs(T, n, D, gamma=True, x_post=True, seed=n + D)
    x = to_dev(bi.x, dev)
    ck = mhc.mhc_checkpoint(x)
    pool = torch.zeros(ck.scales.numel() + 8, dtype=torch.uint8, device=dev)
    at = pool[shift:shift + ck.scales.numel()].view(ck.scales.shape)
    moved = mhc.mhc_checkpoint(x, out=mhc.Checkpoint(torch.empty_like(ck.codes), at, ck.dtype))
    assert torch.equal(moved.scales, ck.scales) and torch.equal(moved.codes, ck.codes)
    assert not pool[:shift].any() and not pool[shift + ck.scales.numel():].any()
    assert torch.equal(mhc.mhc_checkpoint_restore(moved), mhc.mhc_checkpoint_restore(ck))
    args = [to_dev(t, dev) for t in (bi.phi, bi.alpha, bi.grad_h_in, bi.grad_h_post, bi.grad_h_res, bi.inv_rms, bi.h_mix, bi.h_pre, bi.h_post,
                                     bi.gamma, bi.grad_x_post)]
    a, b = (mhc.mhc_pre_backward(c, *args, hc_eps=bi.hc_eps) for c in (ck, moved))
    assert all(torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)) for k in a)
    g = torch.Generator(device=dev).manual_seed(1)
    y, comb = torch.randn(T, D, generator=g, device=dev).to(x.dtype), torch.rand(T, n, n, generator=g, device=dev)
    a, b = (mhc.mhc_post_backward(x, y, c, args[7], comb) for c in (ck, moved))
    assert all(torch.equal(a[k], b[k]) for k in a)
