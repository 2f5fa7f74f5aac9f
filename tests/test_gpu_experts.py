"""The products with 4-bit weights on the GPU against the definition in 64 bits.

Where codes and scale bytes are such that every partial sum is a whole number of a quantum and within 2^24 of them, fp32 sums are
exact in any order, and results are the correctly rounded ones, bit for bit (of the weighted sum in fp16: bf16's terms are first
rounded to 11 bits). Else a sum of K products whose magnitudes add up
to A is off by experts_helpers.sum_error(K, A), and the gated projection's h, with eg and eu for g and u, by 1.13 eg |u| +
|act(g)| eu + 2^-21 |h| before its rounding (|act'| is at most 1.13; 2^-21 for the exponential, the reciprocal and the
products). The weighted sum of k terms adds k 2^-24 of their magnitudes, and in bf16 each term has been rounded to fp16 under the power
of two that takes the largest of 32 to [2^14, 2^15): by 2^-11 of itself, or half of fp16's least step, 2^-25, under that power: 2^-39 of
the largest of 32 at most."""
import sys

import numpy as np
import pytest

from experts_helpers import U, act_ref, check, mxfp4, plan, rounded, sum_error, to_16, to_mxfp4, torch_dtype, values
from gpu_helpers import device

pytestmark = pytest.mark.gpu


def to_dev(a, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def some_experts(rng, T, k, E, masked):
    e = np.stack([rng.permutation(E)[:k] if k <= E else rng.integers(0, E, k) for _ in range(T)]).reshape(T, k).astype(np.int32)
    if masked:
        e[rng.random(T) < 0.25] = -1
        e[rng.random((T, k)) < 0.1] = -1
    return e


def a_plan(e, E, dev):
    import mhc_hyper_connection_amd as mhc
    o, p = plan(e, E)
    return mhc.ExpertsPlan(to_dev(o, dev), to_dev(p, dev), e.shape)


def part_error(v):
    """What rounding the pairs' results v [P, D] to 16 bits adds, at most."""
    P, D = v.shape
    b = np.pad(np.abs(v), ((0, 0), (0, -D % 32))).reshape(P, -1, 32).max(-1)
    return 2.0 ** -11 * np.abs(v) + 2.0 ** -39 * np.repeat(b, 32, -1)[:, :D]


def is_exact(x, w, quantum, K):
    # sums of |terms| within 2^24 quanta
    return (np.abs(x).max() * np.abs(w).max() * K) <= 2 ** 24 * quantum


PRODUCTS = [(1, 1, 8), (1, 7168, 40), (2, 33, 16), (3, 64, 24), (15, 100, 72), (16, 128, 8), (17, 129, 32), (31, 256, 264), (32, 511, 40), (33, 520, 64), (48, 257, 1000),
            (64, 384, 136), (65, 640, 40), (100, 1000, 200), (128, 256, 128), (129, 2056, 136), (255, 500, 256), (300, 768, 520), (700, 96, 1032), (1003, 333, 72),
            (2100, 1024, 1544)]


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("T,K,N", PRODUCTS)
def test_product(T, K, N, f16):
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    rng = np.random.default_rng(T + K + N)
    print(f"[case] product T={T} K={K} N={N} f16={f16}", file=sys.stderr, flush=True)
    # exact: scales 1 and 2, so that products are multiples of 1/4 up to 144
    x, w = mxfp4(rng, T, K, low=127, high=129), mxfp4(rng, N, K, low=127, high=129)
    xv, wv = values(*x, K), values(*w, K)
    full = torch.full((T + 1, N), 7.0, dtype=torch_dtype(f16), device=dev)
    y = mhc.mhc_mxfp4_product(to_mxfp4(*x, K, f16, dev), to_mxfp4(*w, K, f16, dev), out=full[:T])
    want = xv @ wv.T
    if is_exact(xv, wv, 0.25, K):
        assert torch.equal(y.cpu(), torch.from_numpy(want.astype(np.float32)).to(torch_dtype(f16)))
    check("y", y, want, sum_error(K, np.abs(xv) @ np.abs(wv).T), f16)
    assert (full[T] == 7.0).all()
    # values as they come, x in 16 bits
    x16 = to_16(rng.standard_normal((T, K)) * np.exp(0.5 * rng.standard_normal(K)), f16)
    w16 = to_16(rng.standard_normal((N, K)) / np.sqrt(K), f16)
    w4 = mhc.mhc_mxfp4(w16.to(dev))
    xv, wv = rounded(x16.double().numpy(), f16), rounded(w16.double().numpy(), f16)
    y = mhc.mhc_mxfp4_product(x16.to(dev), w4)
    check("y", y, xv @ wv.T, sum_error(K, np.abs(xv) @ np.abs(wv).T), f16)
    again = mhc.mhc_mxfp4_product(mhc.mhc_mxfp4(x16.to(dev)), w4)
    assert torch.equal(again, y)


GROUPED = [(1, 1, 1, 8, 8), (1, 8, 16, 264, 40), (1, 2, 4, 2056, 264), (2, 3, 8, 40, 24), (5, 4, 4, 136, 72), (7, 2, 3, 1000, 136), (16, 8, 64, 128, 64), (33, 6, 9, 200, 72),
           (64, 4, 8, 520, 40), (100, 2, 4, 96, 264), (200, 1, 3, 256, 136), (150, 8, 8, 264, 200), (300, 2, 2, 72, 520), (513, 4, 5, 640, 264), (1003, 3, 4, 136, 72),
           (90, 32, 40, 64, 48), (3, 5, 1024, 32, 16), (260, 2, 200, 40, 40)]


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("T,k,E,D,F", GROUPED)
def test_experts(T, k, E, D, F, f16):
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    dt = torch_dtype(f16)
    rng = np.random.default_rng(T + k + E + D + F)
    e = some_experts(rng, T, k, E, masked=T > 2)
    p = a_plan(e, E, dev)
    flat, tok = e.reshape(-1), np.arange(T * k) // k
    # --- the gated projection
    wg, wu = mxfp4(rng, E, F, D, low=121, high=125), mxfp4(rng, E, F, D, low=121, high=125)
    gv, uv = values(*wg, D), values(*wu, D)
    x16 = to_16(rng.standard_normal((T, D)) * np.exp(0.5 * rng.standard_normal(D)), f16)
    xv = rounded(x16.double().numpy(), f16)
    g, u, ag, au = (np.zeros((T * k, F)) for _ in range(4))
    for x in np.unique(flat[flat >= 0]):
        at = flat == x
        g[at], u[at] = xv[tok[at]] @ gv[x].T, xv[tok[at]] @ uv[x].T
        ag[at], au[at] = np.abs(xv[tok[at]]) @ np.abs(gv[x]).T, np.abs(xv[tok[at]]) @ np.abs(uv[x]).T
    eg, eu = sum_error(D, ag), sum_error(D, au)
    gate, up = to_mxfp4(*wg, D, f16, dev), to_mxfp4(*wu, D, f16, dev)
    for act in ("silu", "gelu_tanh"):
        print(f"[case] experts_glu T={T} k={k} E={E} D={D} F={F} f16={f16} {act}", file=sys.stderr, flush=True)
        a = act_ref(g, act)
        full = torch.full((T + 1, k, F), 7.0, dtype=dt, device=dev)
        h = mhc.mhc_experts_glu(x16.to(dev), p, gate, up, act=act, out=full[:T])
        check("h", h.reshape(T * k, F), a * u, 1.13 * eg * np.abs(u) + np.abs(a) * eu + 2.0 ** -21 * np.abs(a * u), f16)
        assert (full[T] == 7.0).all()
        assert (h.reshape(T * k, F)[to_dev(flat < 0, dev)] == 0).all()
        assert torch.equal(mhc.mhc_experts_glu(mhc.mhc_mxfp4(x16.to(dev)), p, gate, up, act=act), h)
    # --- the projection back
    print(f"[case] experts_down T={T} k={k} E={E} D={D} F={F} f16={f16}", file=sys.stderr, flush=True)
    wd = mxfp4(rng, E, D, F, low=121, high=125)
    dv = values(*wd, F)
    h16 = to_16(rng.standard_normal((T, k, F)), f16)
    hv = rounded(h16.double().numpy(), f16).reshape(T * k, F)
    weights = np.where(e < 0, 0, rng.random((T, k))).astype(np.float32)
    y, mag = np.zeros((T * k, D)), np.zeros((T * k, D))
    for x in np.unique(flat[flat >= 0]):
        at = flat == x
        y[at], mag[at] = hv[at] @ dv[x].T, np.abs(hv[at]) @ np.abs(dv[x]).T
    wt = weights.astype(float).reshape(T * k, 1)
    err = sum_error(F, mag)
    if not f16:
        err = err + part_error(np.abs(y) + err)
    lim = (wt * err).reshape(T, k, D).sum(1) + (k + 1) * U * (wt * np.abs(y)).reshape(T, k, D).sum(1)
    want = (wt * y).reshape(T, k, D).sum(1)
    down = to_mxfp4(*wd, F, f16, dev)
    full = torch.full((T + 1, D), 7.0, dtype=dt, device=dev)
    got = mhc.mhc_experts_down(h16.to(dev), p, to_dev(weights, dev), down, out=full[:T])
    check("y", got, want, lim, f16)
    assert (full[T] == 7.0).all()
    assert torch.equal(mhc.mhc_experts_down(mhc.mhc_mxfp4(h16.to(dev)), p, to_dev(weights, dev), down), got)


@pytest.mark.parametrize("E,loads", [(3, [700, 0, 5]), (5, [0, 0, 0, 0, 0]), (2, [1, 900]), (7, [64, 65, 128, 129, 256, 257, 31]), (4, [17, 16, 0, 300]),
                                     (70, [3] * 69 + [500])])
def test_exact_sums_with_uneven_loads(E, loads):
    # whole numbers: every shape of unit, bit for bit, and the pairs without an expert
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    rng = np.random.default_rng(E)
    e = np.concatenate([np.full(n, x) for x, n in enumerate(loads)] + [np.full(23, -1)]).astype(np.int32)
    e = rng.permutation(e).reshape(-1, 1)
    T, F, D = len(e), 264, 136
    p = a_plan(e, E, dev)
    h, w = mxfp4(rng, T, 1, F, low=127, high=129), mxfp4(rng, E, D, F, low=127, high=129)
    hv, wv = values(*h, F).reshape(T, F), values(*w, F)
    assert is_exact(hv, wv, 0.25, F)
    print(f"[case] loads {loads[:8]}", file=sys.stderr, flush=True)
    want = np.stack([hv[t] @ wv[x].T if x >= 0 else np.zeros(D) for t, x in enumerate(e[:, 0])])
    ones = torch.ones((T, 1), device=dev)
    y = mhc.mhc_experts_down(to_mxfp4(*h, F, True, dev), p, ones, to_mxfp4(*w, F, True, dev))
    assert torch.equal(y.cpu(), torch.from_numpy(want.astype(np.float32)).to(torch.float16))
    y = mhc.mhc_experts_down(to_mxfp4(*h, F, False, dev), p, ones, to_mxfp4(*w, F, False, dev))
    check("y", y, want, part_error(want), False)


@pytest.mark.parametrize("T,E", [(3, 2), (70, 3), (900, 2)])
def test_results_of_any_size_in_bf16(T, E):
    # results far past fp16's range, and neighbours far smaller; an infinite and a NaN one
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    rng = np.random.default_rng(T)
    F, D, k = 64, 200, 2
    e = some_experts(rng, T, k, E, masked=False)
    h, w = mxfp4(rng, T, k, F, low=127, high=129), mxfp4(rng, E, D, F, low=127, high=129)
    # a row's power of two: in the first columns to 2^60 apart, then even, then near the ends of fp32's range
    up = np.concatenate([rng.integers(-30, 31, 96), np.zeros(32), np.full(36, 110), np.full(36, -115)]).astype(int)
    w[1][..., :2] = np.clip(w[1][..., :2].astype(int) + up[None, :, None], 0, 254)
    h[1][0, 0, 0] = 255
    hv, wv = values(*h, F).reshape(T * k, F), values(*w, F)
    flat = e.reshape(-1)
    y, mag = np.zeros((T * k, D)), np.zeros((T * k, D))
    for x in range(E):
        y[flat == x], mag[flat == x] = hv[flat == x] @ wv[x].T, np.abs(hv[flat == x]) @ np.abs(wv[x]).T
    wt = rng.random((T, k)).astype(np.float32)
    print(f"[case] any size T={T} E={E}", file=sys.stderr, flush=True)
    got = mhc.mhc_experts_down(to_mxfp4(*h, F, False, dev), a_plan(e, E, dev), to_dev(wt, dev), to_mxfp4(*w, F, False, dev))
    wd = wt.astype(float).reshape(T * k, 1)
    err = sum_error(F, mag)
    err = err + part_error(np.abs(y) + err) + 2.0 ** -149
    lim = (wd * err).reshape(T, k, D).sum(1) + (k + 1) * U * (wd * np.abs(y)).reshape(T, k, D).sum(1)
    check("y", got, (wd * y).reshape(T, k, D).sum(1), lim, False)


def test_nan_and_infinity_stay_in_their_rows():
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    for T in (5, 40, 300):
        print(f"[case] nan T={T}", file=sys.stderr, flush=True)
        x = torch.randn(T, 200, device=dev).to(torch.bfloat16)
        w = mhc.mhc_mxfp4((torch.randn(72, 200, device=dev) / 14).to(torch.bfloat16))
        clean = mhc.mhc_mxfp4_product(x, w)
        bad = x.clone()
        bad[3, 77] = float("nan")
        bad[1, 199] = -float("inf")
        y = mhc.mhc_mxfp4_product(bad, w)
        assert torch.isnan(y[3]).all() and torch.isnan(y[1]).all()
        rest = [t for t in range(T) if t not in (1, 3)]
        assert torch.equal(y[rest], clean[rest])
        s = w.scales.clone()
        s[5, 2] = 255
        y = mhc.mhc_mxfp4_product(x, w._replace(scales=s))
        assert torch.isnan(y[:, 5]).all() and torch.equal(y[:, 6:], clean[:, 6:]) and torch.equal(y[:, :5], clean[:, :5])
    # a NaN weight of a token, with and without experts
    e = np.array([[0, 1], [1, -1], [-1, -1], [0, 1]], np.int32)
    p = a_plan(e, 2, dev)
    h, wd = torch.randn(4, 2, 64, device=dev).to(torch.bfloat16), mhc.mhc_mxfp4(torch.randn(2, 16, 64, device=dev).to(torch.bfloat16))
    wt = torch.full((4, 2), 0.5, device=dev)
    wt[1, 1] = wt[2, 0] = float("nan")
    y = mhc.mhc_experts_down(h, p, wt, wd)
    assert torch.isnan(y).any(-1).tolist() == [False, True, True, False]


def test_a_plan_that_is_none():
    # offsets and pairs of any content: nothing is read through them, and what they do name is computed
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    T, k, E, D, F = 40, 2, 4, 64, 40
    x = torch.randn(T, D, device=dev).to(torch.bfloat16)
    w = mhc.mhc_mxfp4(torch.randn(E, F, D, device=dev).to(torch.bfloat16))
    rng = np.random.default_rng(1)
    for kind in range(4):
        o = np.array([0, 20, 40, 60, 80], np.int32)
        p = np.arange(T * k, dtype=np.int32)
        if kind == 0:
            o = np.array([-5, 1 << 30, -(1 << 31), 7, 3], np.int32)
        elif kind == 1:
            p = rng.integers(-(1 << 31), (1 << 31) - 1, T * k).astype(np.int32)
        elif kind == 2:
            o = o[::-1].copy()
        else:
            p[::3] = -1
            p[1::3] = T * k
        print(f"[case] plan of any content {kind}", file=sys.stderr, flush=True)
        out = torch.full((T, k, F), 7.0, dtype=torch.bfloat16, device=dev)
        mhc.mhc_experts_glu(x, mhc.ExpertsPlan(to_dev(o, dev), to_dev(p, dev), (T, k)), w, w, out=out)
        torch.cuda.synchronize()
        if kind == 3:
            good = mhc.mhc_experts_glu(x, mhc.ExpertsPlan(to_dev(o, dev), to_dev(np.arange(T * k, dtype=np.int32), dev), (T, k)), w, w)
            named = torch.zeros(T * k, dtype=torch.bool, device=dev)
            named[2::3] = True
            flat = out.reshape(T * k, F)
            assert torch.equal(flat[named], good.reshape(T * k, F)[named]) and (flat[~named] == 7).all()


def test_empty_calls_and_leading_dimensions():
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    w = mhc.mhc_mxfp4(torch.randn(24, 96, device=dev).to(torch.bfloat16))
    x = torch.randn(2, 3, 96, device=dev).to(torch.bfloat16)
    y = mhc.mhc_mxfp4_product(x, w)
    assert y.shape == (2, 3, 24) and torch.equal(y.reshape(6, 24), mhc.mhc_mxfp4_product(x.reshape(6, 96), w))
    assert torch.equal(mhc.mhc_mxfp4_product(x[1, 2].contiguous(), w), y[1, 2])
    assert mhc.mhc_mxfp4_product(x[:0], w).shape == (0, 3, 24)
    E, k = 4, 2
    wg = mhc.mhc_mxfp4(torch.randn(E, 40, 96, device=dev).to(torch.bfloat16))
    wd = mhc.mhc_mxfp4(torch.randn(E, 96, 40, device=dev).to(torch.bfloat16))
    weights, experts = mhc.mhc_route(torch.randn(2, 3, E, device=dev), k)
    p = mhc.mhc_experts_plan(experts, E)
    h = mhc.mhc_experts_glu(x, p, wg, wg)
    y = mhc.mhc_experts_down(h, p, weights, wd)
    assert h.shape == (2, 3, k, 40) and y.shape == (2, 3, 96)
    p6 = p._replace(shape=(6, k))
    h6 = mhc.mhc_experts_glu(x.reshape(6, 96), p6, wg, wg)
    assert torch.equal(h6.reshape(h.shape), h) and torch.equal(mhc.mhc_experts_down(h6, p6, weights.reshape(6, k), wd).reshape(y.shape), y)
    p0 = mhc.mhc_experts_plan(experts[:0], E)
    h0 = mhc.mhc_experts_glu(x[:0], p0, wg, wg)
    assert h0.shape == (0, 3, k, 40) and mhc.mhc_experts_down(h0, p0, weights[:0], wd).shape == (0, 3, 96)


def test_weights_past_32_bits():
    # the last expert's codes lie past 2^32 bytes
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    E, F, D, k = 70, 8192, 16384, 2
    kb, sb = D // 2, D // 32
    print(f"[case] experts past 32 bits E={E} F={F} D={D}", file=sys.stderr, flush=True)
    codes = torch.zeros((E, F, kb), dtype=torch.uint8, device=dev)
    scales = torch.full((E, F, sb), 127, dtype=torch.uint8, device=dev)
    gen = torch.Generator().manual_seed(3)
    some = lambda *s: torch.randint(0, 256, s, generator=gen).to(torch.uint8).to(dev)      # exact sums: multiples of 1/4 up to 36 D
    one = mhc.Mxfp4(some(1, F, kb), scales[:1], torch.bfloat16, D)
    codes[E - 1] = one.codes[0]
    w = mhc.Mxfp4(codes, scales, torch.bfloat16, D)
    for T in (3, 200):
        x = mhc.Mxfp4(some(T, kb), torch.full((T, sb), 127, dtype=torch.uint8, device=dev), torch.bfloat16, D)
        e = np.full((T, k), E - 1, np.int32)
        e[:, 1] = 0
        h = mhc.mhc_experts_glu(x, a_plan(e, E, dev), w, w)
        h1 = mhc.mhc_experts_glu(x, a_plan(np.stack([np.zeros(T), np.full(T, -1)], 1).astype(np.int32), 1, dev), one, one)
        assert torch.equal(h[:, 0], h1[:, 0]) and (h[:, 1] == 0).all() and (h1[:, 0] != 0).any()
