"""Routing to experts on the GPU against the definition in 64 bits. The experts and the plan are whole numbers and equal. A
weight is fp64 until its one rounding to fp32 (2^-24 of it; fp64's own error is 2^-40 at most here); the gradient's error is
derived in experts_helpers.route_backward, with half a step of the logits' format on top."""
import sys

import numpy as np
import pytest

from experts_helpers import U, half_step, plan, route, route_backward
from gpu_helpers import device

pytestmark = pytest.mark.gpu
DT = ["float32", "bfloat16", "float16"]


def make(T, E, seed, dtype, masked=True, spread=1.5):
    import torch
    rng = np.random.default_rng(seed)
    L = spread * rng.standard_normal((T, E))
    if masked:
        L[rng.random((T, E)) < 0.15] = -np.inf
        L[rng.random(T) < 0.2] = -np.inf                 # padded tokens
        for t in range(0, T, 5):                         # tokens with few experts left
            L[t, rng.permutation(E)[:max(0, E - 3)]] = -np.inf
        L[rng.random((T, E)) < 0.02] = 1.25              # equal logits
    L = torch.from_numpy(L.astype(np.float32)).to(getattr(torch, dtype))
    bias = torch.from_numpy((np.round(rng.standard_normal(E) * 50) / 1000).astype(np.float32))
    return L, bias


def check_grad(got, want, lim, dtype):
    got = got.double().cpu().numpy()
    assert (np.isnan(got) == np.isnan(want)).all()
    ok = ~np.isnan(want)
    half = np.maximum(U * np.abs(want), 2.0 ** -150) if dtype == "float32" else half_step(np.abs(want) + lim, dtype == "float16")
    err = np.abs(got - want)
    lim = lim + half + 1e-12 * np.abs(want)
    assert (err[ok] <= lim[ok]).all(), (float((err[ok] / lim[ok]).max()), np.argwhere(~(err <= lim) & ok)[:4].tolist())


def run(L, bias, k, dev, dtype, seed, **kw):
    import mhc_hyper_connection_amd as mhc
    import torch
    T, E = L.shape
    g = L.to(dev)
    fw = {a: b for a, b in kw.items()}
    full = (torch.full((T + 1, k), 7.0, device=dev), torch.full((T + 1, k), 7, dtype=torch.int32, device=dev))
    w, e = mhc.mhc_route(g, k, bias=None if bias is None else bias.to(dev), out=(full[0][:T], full[1][:T]), **fw)
    Ld = L.double().numpy()
    ww, we = route(Ld, k, None if bias is None else bias.double().numpy(), **kw)
    assert np.array_equal(e.cpu().numpy(), we), np.argwhere(e.cpu().numpy() != we)[:4].tolist()
    got = w.double().cpu().numpy()
    assert (np.isnan(got) == np.isnan(ww)).all()
    ok = ~np.isnan(ww)
    assert (np.abs(got - ww)[ok] <= (np.maximum(U * np.abs(ww), 2.0 ** -150) * (1 + 2.0 ** -16))[ok]).all()
    assert (full[0][T] == 7).all() and (full[1][T] == 7).all()      # the row behind the last token stays as it was
    p = mhc.mhc_experts_plan(e, E)
    po, pp = plan(we, E)
    assert np.array_equal(p.offsets.cpu().numpy(), po) and np.array_equal(p.pairs.cpu().numpy(), pp)
    assert p.shape == (T, k)
    gw = torch.from_numpy(np.random.default_rng(seed + 1).standard_normal((T, k)).astype(np.float32)).to(dev)
    back = {a: b for a, b in kw.items() if a in ("score", "renormalise", "scale")}
    guard = torch.full((T + 1, E), 7.0, dtype=g.dtype, device=dev)
    d = mhc.mhc_route_backward(gw, g, w, e, out=guard[:T], **back)
    want, lim = route_backward(gw.double().cpu().numpy(), Ld, got, we, **back)
    check_grad(d, want, lim, dtype)
    assert (guard[T] == 7).all()


SIZES = [(1, 1, 1), (1, 128, 8), (3, 2, 2), (17, 60, 4), (16, 64, 16), (33, 65, 5), (5, 128, 32), (64, 100, 7), (130, 256, 8), (9, 255, 31), (12, 257, 9),
         (7, 512, 10), (5, 513, 32), (6, 1000, 22), (4, 1024, 1)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,E,k", SIZES)
def test_sizes(T, E, k, dtype, score):
    dev = device()
    for n, (biased, renorm, scale) in enumerate(((False, True, 1.0), (True, True, 2.5), (True, False, 1.0), (False, False, 0.25))):
        print(f"[case] route T={T} E={E} k={k} {dtype} {score} bias={biased} renorm={renorm}", file=sys.stderr, flush=True)
        L, bias = make(T, E, T + E + n, dtype, masked=n % 2 == 0)
        run(L, bias if biased else None, k, dev, dtype, n, score=score, renormalise=renorm, scale=scale)


@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top_groups,k", [(8, 8, 3, 3), (16, 2, 1, 8), (60, 4, 2, 9), (256, 8, 4, 8), (112, 16, 5, 6), (500, 4, 3, 32), (1024, 16, 16, 8),
                                                   (1024, 2, 1, 20)])
def test_groups(E, groups, top_groups, k, score, biased, group_top):
    dev = device()
    for masked in (False, True):
        print(f"[case] groups E={E} {groups}/{top_groups} k={k} {score} bias={biased} top{group_top} masked={masked}", file=sys.stderr, flush=True)
        L, bias = make(40, E, E + groups, "float32", masked)
        if masked:   # a group of nothing but masked experts, and a masked bias
            L[1::3, :E // groups] = -float("inf")
            bias[E // 2] = -float("inf")
        run(L, bias if biased else None, k, dev, "float32", 3, score=score, groups=groups, top_groups=top_groups, group_top=group_top, scale=2.5)


@pytest.mark.parametrize("near", [1e-9, 3e-8, 1e-6, 3e-5])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many_tokens_and_near_ties(score, near):
    # scores nearer to each other than fp32 tells, or about as near: the order is that of 64 bits
    import torch
    dev = device()
    rng = np.random.default_rng(5)
    T, E = 1501, 64
    L = torch.from_numpy((np.round(rng.standard_normal((T, E)) * 4) / 4).astype(np.float32))
    bias = torch.from_numpy((near * rng.permutation(E)).astype(np.float32))
    for groups, top_groups in ((1, 1), (8, 3)):
        print(f"[case] near ties {score} {near} {groups}", file=sys.stderr, flush=True)
        run(L, bias, 8, dev, "float32", 1, score=score, groups=groups, top_groups=top_groups)


@pytest.mark.parametrize("dtype", DT)
def test_near_logits_without_a_bias(dtype):
    # neighbours in the format, equal ones, zeros of either sign, subnormal ones
    import torch
    dev = device()
    rng = np.random.default_rng(6)
    for unit, offset in ((2.0 ** -22, 1.0), (2.0 ** -18, -2.0), (2.0 ** -149, 0.0), (2.0 ** -24, 0.0), (2.0 ** -7, 1.5), (2.0 ** -10, -1.0)):
        L = torch.from_numpy((offset + unit * rng.integers(-20, 20, (300, 96))).astype(np.float32)).to(getattr(torch, dtype))
        L[::3] = torch.where(L[::3] == 0, -L[::3], L[::3])
        for groups, top_groups in ((1, 1), (4, 2)):
            print(f"[case] near logits {dtype} {unit} {groups}", file=sys.stderr, flush=True)
            run(L, None, 10, dev, dtype, 1, groups=groups, top_groups=top_groups)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_extreme_values(score):
    import torch
    dev = device()
    inf, nan = float("inf"), float("nan")
    rows = [[0, 0, 0, 0], [1e30, -1e30, 0, 1], [-1e30] * 4, [inf, 0, 1, 2], [nan, 0, 1, 2], [-inf] * 4, [-inf, nan, 1, 2], [-inf, -inf, -inf, 3],
            [700, 710, -700, -750], [-800, -900, -1000, -inf], [50, 60, 40, 45], [3e38, 3e38, -3e38, 0], [1e-40, -1e-40, 0, 1e-45]]
    L = torch.tensor(rows)
    for renorm in (True, False):
        for bias in (None, torch.tensor([0.0, -inf, 0.5, 0.0]), torch.tensor([0.0, inf, 0.5, 0.25]), torch.tensor([0.0, nan, 0.5, 0.25])):
            print(f"[case] extreme {score} {renorm} {bias}", file=sys.stderr, flush=True)
            run(L, bias, 3, dev, "float32", 2, score=score, renormalise=renorm)


def test_backward_against_differences():
    # the forward's own formula in 64 bits, differentiated by central differences at fixed experts
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    rng = np.random.default_rng(8)
    T, E, k = 6, 24, 4
    L = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32))
    gw = rng.standard_normal((T, k)).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            w, e = mhc.mhc_route(L.to(dev), k, score=score, renormalise=renorm, scale=1.5)
            got = mhc.mhc_route_backward(torch.from_numpy(gw).to(dev), L.to(dev), w, e, score=score, renormalise=renorm, scale=1.5).cpu().double().numpy()
            at = e.cpu().numpy()

            def loss(x):
                s = np.exp(x) / np.exp(x).sum(-1, keepdims=True) if score == "softmax" else 1 / (1 + np.exp(-x))
                c = s[np.arange(T)[:, None], at]
                return (gw * 1.5 * (c / c.sum(-1, keepdims=True) if renorm else c)).sum(-1)
            x, h = L.double().numpy(), 1e-5
            for i in range(E):
                d = np.zeros((T, E))
                d[:, i] = h
                diff = (loss(x + d) - loss(x - d)) / (2 * h)
                # third derivatives of a few units give h^2 units; differences of values near 1 are off by 2^-52 / h; fp32 by 64 steps
                assert (np.abs(diff - got[:, i]) <= 1e-8 + 64 * U * (1 + np.abs(diff))).all()


def test_the_same_expert_twice_and_no_experts():
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    rng = np.random.default_rng(2)
    T, E, k = 21, 40, 6
    L = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32))
    e = rng.integers(-2, E + 2, (T, k)).astype(np.int32)       # some are no experts
    e[:, 3] = e[:, 1]
    e[::2, 5] = e[::2, 1]
    w = rng.random((T, k)).astype(np.float32)
    gw = rng.standard_normal((T, k)).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            got = mhc.mhc_route_backward(*(torch.from_numpy(a).to(dev) for a in (gw, L.numpy(), w, e)), score=score, renormalise=renorm)
            want, lim = route_backward(gw.astype(float), L.double().numpy(), w.astype(float), e, score=score, renormalise=renorm)
            check_grad(got, want, lim, "float32")
    p = mhc.mhc_experts_plan(torch.from_numpy(e).to(dev), E)
    po, pp = plan(e, E)
    assert np.array_equal(p.offsets.cpu().numpy(), po) and np.array_equal(p.pairs.cpu().numpy(), pp)


@pytest.mark.parametrize("P,E", [(0, 5), (1, 1), (63, 3), (64, 1024), (513, 7), (4096, 256), (4097, 256), (10007, 60), (70001, 1000), (600011, 33)])
def test_plan_sizes(P, E):
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    rng = np.random.default_rng(P + E)
    for kind in range(3):
        e = rng.integers(-1, E, P) if kind == 0 else (np.minimum(rng.geometric(0.2, P) - 1, E - 1) if kind == 1 else np.full(P, E - 1))
        e = e.astype(np.int32)
        print(f"[case] plan P={P} E={E} kind={kind}", file=sys.stderr, flush=True)
        p = mhc.mhc_experts_plan(torch.from_numpy(e).to(dev), E)
        po, pp = plan(e, E)
        assert np.array_equal(p.offsets.cpu().numpy(), po)
        assert np.array_equal(p.pairs.cpu().numpy(), pp)


def test_no_tokens_and_leading_dimensions():
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    w, e = mhc.mhc_route(torch.empty((0, 16), device=dev), 3)
    assert w.shape == e.shape == (0, 3)
    assert mhc.mhc_route_backward(w, torch.empty((0, 16), device=dev), w, e).shape == (0, 16)
    p = mhc.mhc_experts_plan(e, 16)
    assert p.pairs.numel() == 0 and (p.offsets == 0).all()
    L = torch.randn(2, 3, 16, device=dev)
    w, e = mhc.mhc_route(L, 4)
    w2, e2 = mhc.mhc_route(L.reshape(6, 16), 4)
    assert w.shape == (2, 3, 4) and torch.equal(w.reshape(6, 4), w2) and torch.equal(e.reshape(6, 4), e2)
    w1, e1 = mhc.mhc_route(L[1, 2].contiguous(), 4)              # one token without leading dimensions
    assert w1.shape == (4,) and torch.equal(e1, e2[5])
    with pytest.raises(mhc.MhcError):
        mhc.mhc_route(L, 17)
    with pytest.raises(mhc.MhcError):
        mhc.mhc_route(L, 4, groups=3)


def test_rows_at_odd_addresses():
    # 16-bit logits whose rows start at any even address
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    big = torch.randn(12, 61, device=dev).to(torch.bfloat16)
    w, e = mhc.mhc_route(big[1:], 4)
    w2, e2 = mhc.mhc_route(big[1:].clone(), 4)
    assert torch.equal(w, w2) and torch.equal(e, e2)
