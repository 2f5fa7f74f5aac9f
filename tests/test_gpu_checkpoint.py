"""The 8-bit checkpoints on the GPU: codes and scales equal to the definition's (numpy, 64 bits), restored values exact,
hc_post's fused form equal to the two calls, and the pre-mapping's backward from a checkpoint equal, bit for bit, to the
one from the restored tensor. The format is exact arithmetic but for one rounding to an integer, so nothing here has a
tolerance, save the error bound that the format promises."""
import sys

import numpy as np
import pytest

import synth
import test_gpu_backward as tb
from gpu_helpers import device, to_dev, to_host
from train_helpers import BLOCK, load, store, to_16, torch_dtype

pytestmark = pytest.mark.gpu


def values(kind, rows, D, f16, seed):
    """float64 array of 16-bit values."""
    rng = np.random.default_rng(seed)
    a = rng.standard_normal((rows, D))
    if kind == "outliers":
        a *= np.exp(rng.standard_normal(D))
        a[:, rng.random(D) < 0.05] *= 50.0
    elif kind == "wide":          # every magnitude the format has
        lo, hi = (-26, 15.9) if f16 else (-135, 127.9)
        a = np.sign(a) * np.exp2(rng.uniform(lo, hi, (rows, D)))
    elif kind == "tiny":          # the format's least values, and zeros
        a = rng.integers(-3, 4, (rows, D)) * (2.0 ** -24 if f16 else 2.0 ** -133)
    elif kind == "zero":
        a = np.zeros((rows, D))
        a[..., 0] = -0.0
    elif kind == "top":           # the largest finite values beside ties: multiples of half a step
        big = 65504.0 if f16 else float(np.float32(3.3895314e38))
        a = rng.integers(-255, 256, (rows, D)) * (big / 2.0 ** (7 + (0 if f16 else 0)) / 2)
        a[:, ::BLOCK] = big
        a = np.clip(a, -big, big)
    elif kind == "ties":
        a = rng.integers(-255, 256, (rows, D)) * 2.0 ** -8
    return to_16(a, f16).double().numpy()


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("kind", ["normal", "outliers", "wide", "tiny", "zero", "top", "ties"])
def test_format(kind, f16):
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    for rows, D in ((1, 8), (1, 32), (3, 24), (7, 40), (130, 1000), (65, 256), (33, 4096), (5, 16384), (2, 16376)):
        print(f"[case] checkpoint {kind} f16={f16} rows={rows} D={D}", file=sys.stderr, flush=True)
        v = values(kind, rows, D, f16, seed=rows * D)
        x = to_16(v, f16).to(dev)
        ck = mhc.mhc_checkpoint(x)
        assert ck.codes.shape == (rows, D) and ck.scales.shape == (rows, -(-D // BLOCK)) and ck.dtype == x.dtype
        q, s = store(v, f16)
        assert np.array_equal(to_host(ck.codes), q)
        assert np.array_equal(to_host(ck.scales), s)
        back = mhc.mhc_checkpoint_restore(ck).double().cpu().numpy()
        want = load(q, s)
        assert np.array_equal(back, want)
        # half a step (a step above 127.5 steps) of the block's step
        step = np.repeat(np.ldexp(1.0, s.astype(np.int64) - 127), BLOCK, -1)[:, :D]
        off = np.abs(back - v)
        assert (off <= np.where(np.abs(v) > 127.5 * step, step, step / 2)).all()
        assert torch.isfinite(mhc.mhc_checkpoint_restore(ck)).all()


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("D", [64, 40])
def test_blocks_that_are_not_finite(D, f16):
    import mhc_hyper_connection_amd as mhc
    dev = device()
    v = values("normal", 6, D, f16, 3)
    v[1, 5], v[2, 33], v[3, 0] = np.nan, np.inf, -np.inf
    print(f"[case] checkpoint not finite D={D} f16={f16}", file=sys.stderr, flush=True)
    ck = mhc.mhc_checkpoint(to_16(v, f16).to(dev))
    q, s = store(v, f16)
    assert np.array_equal(to_host(ck.scales), s) and np.array_equal(to_host(ck.codes), q)
    back = mhc.mhc_checkpoint_restore(ck).double().cpu().numpy()
    bad = np.zeros_like(v, dtype=bool)
    bad[1, :32] = bad[2, 32:] = bad[3, :32] = True
    assert np.array_equal(np.isnan(back), bad)
    assert np.array_equal(back[~bad], load(q, s)[~bad])


def test_leading_dimensions_empty_and_given_outputs():
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    x = to_16(values("normal", 30, 48, False, 1).reshape(2, 3, 5, 48), False).to(dev)
    print("[case] checkpoint leading dimensions", file=sys.stderr, flush=True)
    ck = mhc.mhc_checkpoint(x)
    assert ck.codes.shape == x.shape and ck.scales.shape == (2, 3, 5, 2)
    into = mhc.Checkpoint(torch.empty_like(ck.codes), torch.empty_like(ck.scales), x.dtype)
    assert mhc.mhc_checkpoint(x, out=into) is into and torch.equal(into.codes, ck.codes)
    out = torch.empty_like(x)
    assert mhc.mhc_checkpoint_restore(ck, out=out) is out
    assert torch.equal(out, mhc.mhc_checkpoint_restore(mhc.Checkpoint(ck.codes.reshape(30, 48), ck.scales.reshape(30, 2), x.dtype)).reshape(x.shape))
    empty = mhc.mhc_checkpoint(torch.empty((0, 4, 64), dtype=torch.float16, device=dev))
    assert empty.codes.shape == (0, 4, 64) and mhc.mhc_checkpoint_restore(empty).shape == (0, 4, 64)


@pytest.mark.parametrize("T,n,D,f16", [(1, 4, 8, False), (3, 4, 40, True), (65, 6, 1000, True), (37, 8, 2048, False),
                                       (300, 4, 7168, False), (5, 8, 16384, True), (1, 6, 24, False)])
def test_post_checkpoint_is_post_and_its_checkpoint(T, n, D, f16):
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    print(f"[case] post_checkpoint T={T} n={n} D={D} f16={f16}", file=sys.stderr, flush=True)
    pi = synth.post_inputs(T, n, D, seed=T + D)
    x, res = (torch.from_numpy(synth.bf16_bits_to_f32(a)).to(torch_dtype(f16)).to(dev) for a in (pi.x, pi.residual))
    post, comb = to_dev(pi.post, dev), to_dev(pi.comb, dev)
    # one value past D of a code row or a scale row would show in the guard rows
    codes = torch.full((T + 1, n, D), 99, dtype=torch.int8, device=dev)
    scales = torch.full((T + 1, n, -(-D // BLOCK)), 99, dtype=torch.uint8, device=dev)
    out, ck = mhc.mhc_post_checkpoint(x, res, post, comb, checkpoint=mhc.Checkpoint(codes[:T], scales[:T], x.dtype))
    want = mhc.mhc_post(x, res, post, comb)
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    two = mhc.mhc_checkpoint(want)
    assert torch.equal(ck.codes, two.codes) and torch.equal(ck.scales, two.scales)
    assert (codes[T] == 99).all() and (scales[T] == 99).all()


@pytest.mark.parametrize("T,n,D,gamma,post,it,f16", [
    (1, 4, 8, False, False, 0, False), (70, 4, 264, True, True, 20, False), (130, 4, 1000, False, True, 3, True),
    (65, 6, 1032, True, False, 20, False), (33, 6, 520, False, True, 0, True), (200, 8, 104, True, True, 2, True),
    (64, 8, 2048, False, False, 20, False), (3, 4, 16384, True, False, 1, True), (513, 4, 7168, False, False, 20, False)])
def test_pre_backward_from_a_checkpoint_is_the_one_from_its_values(T, n, D, gamma, post, it, f16):
    import dataclasses
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    print(f"[case] pre_backward ckpt T={T} n={n} D={D} gamma={gamma} post={post} it={it} f16={f16}", file=sys.stderr, flush=True)
    bi = synth.backward_inputs(T, n, D, gamma=gamma, x_post=post, sinkhorn_iters=it, seed=T + D + n, x_f16=f16)
    ck = mhc.mhc_checkpoint(to_dev(bi.x, dev, f16))
    kept = mhc.mhc_checkpoint_restore(ck)
    args = [to_dev(a, dev, f16) for a in (bi.phi, bi.alpha, bi.grad_h_in, bi.grad_h_post, bi.grad_h_res, bi.inv_rms,
                                          bi.h_mix, bi.h_pre, bi.h_post, bi.gamma, bi.grad_x_post)]
    kw = dict(hc_eps=bi.hc_eps, num_iters=it)
    if it:
        kw.update(sum_out=to_dev(bi.sum_out, dev), norm_out=to_dev(bi.norm_out, dev))
    a, b = mhc.mhc_pre_backward(ck, *args, **kw), mhc.mhc_pre_backward(kept, *args, **kw)
    assert set(a) == set(b)
    for k in a:
        assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k
    # and against the fp64 oracle on the values the checkpoint stands for
    bk = dataclasses.replace(bi, x=to_host(kept))
    rep = tb.compare({k: to_host(v) for k, v in a.items()}, tb.run_oracle(bk), bk)
    assert all(v["fail"] == 0 for v in rep.values()), rep


def test_pre_backward_from_an_empty_checkpoint():
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    n, D = 4, 64
    M = n * n + 2 * n
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device=dev)
    print("[case] pre_backward ckpt T=0", file=sys.stderr, flush=True)
    ck = mhc.mhc_checkpoint(z(0, n, D, dt=torch.bfloat16))
    out = mhc.mhc_pre_backward(ck, z(M, n * D), z(3), z(0, D, dt=torch.bfloat16), z(0, n), z(0, n, n), z(0), z(0, M), z(0, n), z(0, n))
    assert out["grad_x"].shape == (0, n, D) and not out["grad_phi"].any() and not out["grad_alpha"].any()
