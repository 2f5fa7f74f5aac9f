"""The products with 4-bit weights in tiles on the GPU, at sizes for which the launch plan takes them (tests/test_experts_tiles_host.py),
against the definition in 64 bits; the errors are those of tests/test_gpu_experts.py, whose rounding of bf16's terms is that of short_terms alone."""
import sys

import numpy as np
import pytest

from experts_helpers import U, act_ref, check, mxfp4, rounded, sum_error, to_16, to_mxfp4, torch_dtype, values
from experts_tiles import DOWN, FAR, FAR_RESULTS, GLU, PRODUCTS
from gpu_helpers import device
from test_gpu_experts import a_plan, is_exact, part_error, some_experts, to_dev

pytestmark = pytest.mark.gpu


def case(text):
    print(f"[case] {text}", file=sys.stderr, flush=True)


def pairs_of(x, w, flat, tok):
    """x[tok[p]] w[flat[p]]^T for each pair p with an expert, zeros for the others."""
    out = np.zeros((len(flat), w.shape[1]))
    for e in np.unique(flat[flat >= 0]):
        at = flat == e
        out[at] = x[tok[at]] @ w[e].T
    return out


FORMS = [(False, False), (False, True), (True, False), (True, True)]      # f16, short_terms


@pytest.mark.parametrize("f16,short", FORMS)
@pytest.mark.parametrize("T,k,E,D,F,shape", DOWN)
def test_finite_results_beside_a_nan_or_an_infinity(T, k, E, D, F, shape, f16, short):
    # A weight row with a block of NaN spoils its column of y for its expert's tokens, and one whose sums overflow makes them
    # infinite; the columns beside them are those of weights without either. Whole numbers, whose fp32 sums are exact.
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    rng = np.random.default_rng(T + D)
    case(f"finite beside NaN T={T} k={k} E={E} D={D} F={F} f16={f16} short={short}")
    e = some_experts(rng, T, k, E, masked=True)
    flat = e.reshape(-1)
    h, w = mxfp4(rng, T, k, F, low=127, high=129), mxfp4(rng, E, D, F, low=127, high=129)
    h[0][..., 0] = h[0][..., 0] & 0xF0 | 7                   # 6 at the first place
    nan, inf = [37, D - 3], [44, D - 7]                      # two in one run of 32 each; the last run is short
    w[0][0, nan] = w[0][1, inf] = 0
    wt = (1 + rng.integers(0, 4, (T, k))).astype(np.float32) / 4
    p, hm, wd = a_plan(e, E, dev), to_mxfp4(*h, F, f16, dev), to_dev(wt, dev)
    clean = mhc.mhc_experts_down(hm, p, wd, to_mxfp4(*w, F, f16, dev), short_terms=short)
    hv, wv = values(*h, F).reshape(T * k, F), values(*w, F)
    y = pairs_of(hv, wv, flat, np.arange(T * k))
    err = part_error(y) if short and not f16 else np.zeros_like(y)
    weighted = lambda v: (wt.astype(float).reshape(T * k, 1) * v).reshape(T, k, D).sum(1)
    check("clean", clean, weighted(y), weighted(err) + (k + 1) * U * weighted(np.abs(y)), f16)

    w[1][0, nan, 1] = 255                                    # a block of the reduction's second 32 values
    w[0][1, inf, 0], w[1][1, inf, 0] = 7, 254                # 6 2^127 6 2^0, or 2^1, is past fp32's range
    got = mhc.mhc_experts_down(hm, p, wd, to_mxfp4(*w, F, f16, dev), short_terms=short).cpu()
    clean = clean.cpu()
    has = lambda x: torch.from_numpy((e == x).any(1))
    rest = torch.ones(D, dtype=torch.bool)
    rest[nan + inf] = False
    assert has(0).any() and has(1).any() and (~has(0)).any() and (~has(1)).any()
    assert torch.equal(got[:, rest], clean[:, rest])
    assert torch.isnan(got[:, nan][has(0)]).all() and torch.equal(got[:, nan][~has(0)], clean[:, nan][~has(0)])
    assert (got[:, inf][has(1)] == float("inf")).all() and torch.equal(got[:, inf][~has(1)], clean[:, inf][~has(1)])


def uneven(rng, T, k, E):
    """Experts [T, k]: an expert with most of the pairs, one with a few, one with none (where there are three), and pairs without one."""
    share = np.array([0.62, 0.0 if E > 2 else 0.01, 0.01, *[0.1] * (E - 3)][:E])
    p = np.concatenate([share, [1 - share.sum()]])
    return np.concatenate([np.arange(E), [-1]])[rng.choice(E + 1, (T, k), p=p)].astype(np.int32)


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("T,K,N,shape", PRODUCTS)
def test_product(T, K, N, shape, f16):
    # whole numbers bit for bit; values as they come, x in 16 bits and in 4; and the rows and columns of a NaN or an infinity alone
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    rng = np.random.default_rng(T + K + N)
    case(f"product T={T} K={K} N={N} f16={f16}")
    x, w = mxfp4(rng, T, K, low=127, high=129), mxfp4(rng, N, K, low=127, high=129)
    xv, wv = values(*x, K), values(*w, K)
    assert is_exact(xv, wv, 0.25, K)
    full = torch.full((T + 1, N), 7.0, dtype=torch_dtype(f16), device=dev)
    y = mhc.mhc_mxfp4_product(to_mxfp4(*x, K, f16, dev), to_mxfp4(*w, K, f16, dev), out=full[:T])
    assert torch.equal(y.cpu(), torch.from_numpy((xv @ wv.T).astype(np.float32)).to(torch_dtype(f16)))
    assert (full[T] == 7.0).all()

    x16 = to_16(rng.standard_normal((T, K)) * np.exp(0.5 * rng.standard_normal(K)), f16)
    w4 = mhc.mhc_mxfp4(to_16(rng.standard_normal((N, K)) / np.sqrt(K), f16).to(dev))
    xv, wv = rounded(x16.double().numpy(), f16), values(w4.codes.cpu().numpy(), w4.scales.cpu().numpy(), K)
    y = mhc.mhc_mxfp4_product(x16.to(dev), w4)
    check("y", y, xv @ wv.T, sum_error(K, np.abs(xv) @ np.abs(wv).T), f16)
    assert torch.equal(mhc.mhc_mxfp4_product(mhc.mhc_mxfp4(x16.to(dev)), w4), y)

    bad = x16.clone()
    bad[3, K // 2], bad[T - 1, K - 1] = float("nan"), -float("inf")
    s = w4.scales.clone()
    s[5, 1] = s[N - 2, 0] = 255
    z = mhc.mhc_mxfp4_product(bad.to(dev), w4._replace(scales=s))
    rows, columns = torch.ones(T, dtype=torch.bool, device=dev), torch.ones(N, dtype=torch.bool, device=dev)
    rows[[3, T - 1]] = columns[[5, N - 2]] = False
    assert torch.isnan(z[~rows]).all() and torch.isnan(z[:, ~columns]).all()
    assert torch.equal(z[rows][:, columns], y[rows][:, columns])


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("T,k,E,D,F,shape", GLU)
def test_gated_projection_with_uneven_loads(T, k, E, D, F, shape, f16):
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    rng = np.random.default_rng(T + D + F)
    e = uneven(rng, T, k, E)
    flat, tok, p = e.reshape(-1), np.arange(T * k) // k, a_plan(e, E, dev)
    wg, wu = mxfp4(rng, E, F, D, low=121, high=125), mxfp4(rng, E, F, D, low=121, high=125)
    gv, uv = values(*wg, D), values(*wu, D)
    x16 = to_16(rng.standard_normal((T, D)) * np.exp(0.5 * rng.standard_normal(D)), f16)
    xv = rounded(x16.double().numpy(), f16)
    g, u = pairs_of(xv, gv, flat, tok), pairs_of(xv, uv, flat, tok)
    eg, eu = (sum_error(D, pairs_of(np.abs(xv), np.abs(v), flat, tok)) for v in (gv, uv))
    gate, up = to_mxfp4(*wg, D, f16, dev), to_mxfp4(*wu, D, f16, dev)
    for act in ("silu", "gelu_tanh"):
        case(f"experts_glu T={T} k={k} E={E} D={D} F={F} f16={f16} {act}")
        a = act_ref(g, act)
        full = torch.full((T + 1, k, F), 7.0, dtype=torch_dtype(f16), device=dev)
        h = mhc.mhc_experts_glu(x16.to(dev), p, gate, up, act=act, out=full[:T])
        check("h", h.reshape(T * k, F), a * u, 1.13 * eg * np.abs(u) + np.abs(a) * eu + 2.0 ** -21 * np.abs(a * u), f16)
        assert (full[T] == 7.0).all() and (h.reshape(T * k, F)[to_dev(flat < 0, dev)] == 0).all()
        assert torch.equal(mhc.mhc_experts_glu(mhc.mhc_mxfp4(x16.to(dev)), p, gate, up, act=act), h)
    # a NaN of a token, and of a row of either weight
    bad = x16.clone()
    bad[3, D // 2] = float("nan")
    bg, bu = gate.scales.clone(), up.scales.clone()
    bg[0, 5, 1] = bu[0, F - 2, 0] = 255
    z = mhc.mhc_experts_glu(bad.to(dev), p, gate._replace(scales=bg), up._replace(scales=bu), act=act).cpu()
    nan = torch.zeros(T, k, F, dtype=torch.bool)
    nan[3] = True
    first = torch.from_numpy(e == 0)
    nan[..., 5] |= first
    nan[..., F - 2] |= first
    nan[torch.from_numpy(e < 0)] = False
    assert first.any() and torch.equal(torch.isnan(z), nan) and torch.equal(z[~nan], h.cpu()[~nan])


@pytest.mark.parametrize("T,k,E,D,F,shape", DOWN)
def test_projection_back_with_uneven_loads(T, k, E, D, F, shape):
    # whole numbers: the terms bit for bit (one slot of weight 1), then weighted sums; both forms of h
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    rng = np.random.default_rng(T + D + F)
    e = uneven(rng, T, k, E)
    flat, p = e.reshape(-1), a_plan(e, E, dev)
    w = mxfp4(rng, E, D, F, low=127, high=129)
    wv = values(*w, F)
    h = mxfp4(rng, T, k, F, low=127, high=129)
    hv = values(*h, F).reshape(T * k, F)
    assert is_exact(hv, wv, 0.25, F)
    y = pairs_of(hv, wv, flat, np.arange(T * k))
    alone = np.zeros((T, k), np.float32)
    alone[np.arange(T), rng.integers(0, k, T)] = 1
    some = np.where(e < 0, 0, rng.random((T, k))).astype(np.float32)
    for f16, short in FORMS:
        case(f"experts_down T={T} k={k} E={E} D={D} F={F} f16={f16} short={short}")
        rounds = short and not f16
        err = part_error(y) if rounds else np.zeros_like(y)
        wd, hm = to_mxfp4(*w, F, f16, dev), to_mxfp4(*h, F, f16, dev)
        for wt in (alone, some):
            weighted = lambda v: (wt.astype(float).reshape(T * k, 1) * v).reshape(T, k, D).sum(1)
            full = torch.full((T + 1, D), 7.0, dtype=torch_dtype(f16), device=dev)
            got = mhc.mhc_experts_down(hm, p, to_dev(wt, dev), wd, short_terms=short, out=full[:T])
            want = weighted(y)
            if not rounds and wt is alone:
                assert torch.equal(got.cpu(), torch.from_numpy(want.astype(np.float32)).to(torch_dtype(f16)))
            check("y", got, want, weighted(err) + (k + 1) * U * weighted(np.abs(y)), f16)
            assert (full[T] == 7.0).all()
        # h in 16 bits whose 4-bit form is h itself
        h16 = mhc.mhc_mxfp4_restore(hm)
        assert torch.equal(*(mhc.mhc_experts_down(v, p, to_dev(some, dev), wd, short_terms=short) for v in (h16, mhc.mhc_mxfp4(h16))))


@pytest.mark.parametrize("short", [False, True])
@pytest.mark.parametrize("T,k,E,D,F,shape", DOWN)
def test_results_of_any_size_in_bf16(T, k, E, D, F, shape, short):
    # a run of 32 results far past fp16's range or far below it, and neighbours 2^60 apart; a pair whose h is NaN
    import mhc_hyper_connection_amd as mhc
    dev = device()
    rng = np.random.default_rng(T)
    case(f"any size T={T} k={k} E={E} D={D} F={F} short={short}")
    e = some_experts(rng, T, k, E, masked=False)
    flat = e.reshape(-1)
    h, w = mxfp4(rng, T, k, F, low=127, high=129), mxfp4(rng, E, D, F, low=127, high=129)
    up = np.concatenate([rng.integers(-30, 31, D - 104), np.zeros(32), np.full(36, 105), np.full(36, -115)]).astype(int)
    nb = -(-F // 32)
    w[1][..., :nb] = np.clip(w[1][..., :nb].astype(int) + up[None, :, None], 0, 254)
    h[1][0, 0, 0] = 255
    hv, wv = values(*h, F).reshape(T * k, F), values(*w, F)
    y, mag = pairs_of(hv, wv, flat, np.arange(T * k)), pairs_of(np.abs(hv), np.abs(wv), flat, np.arange(T * k))
    wt = rng.random((T, k)).astype(np.float32)
    got = mhc.mhc_experts_down(to_mxfp4(*h, F, False, dev), a_plan(e, E, dev), to_dev(wt, dev), to_mxfp4(*w, F, False, dev), short_terms=short)
    weighted = lambda v: (wt.astype(float).reshape(T * k, 1) * v).reshape(T, k, D).sum(1)
    err = sum_error(F, mag)
    err = err + (part_error(np.abs(y) + err) if short else 0) + 2.0 ** -149
    check("y", got, weighted(y), weighted(err) + (k + 1) * U * weighted(np.abs(y)), False)


@pytest.mark.parametrize("kind", range(4))
@pytest.mark.parametrize("T,k,E,D,F,shape", GLU)
def test_a_plan_that_is_none(T, k, E, D, F, shape, kind):
    # offsets and pairs of any content: nothing is read or written through them, and what they do name is computed
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    rng = np.random.default_rng(kind)
    gen = torch.Generator(device=dev).manual_seed(kind)
    randn = lambda *s: torch.randn(*s, device=dev, generator=gen).to(torch.bfloat16)
    P = T * k
    o, q = np.linspace(0, P, E + 1).astype(np.int32), np.arange(P, dtype=np.int32)
    if kind == 0:
        o = rng.integers(-(1 << 31), (1 << 31) - 1, E + 1).astype(np.int32)
    elif kind == 1:
        q = rng.integers(-(1 << 31), (1 << 31) - 1, P).astype(np.int32)
    elif kind == 2:
        o = np.array([P if e % 2 else 0 for e in range(E + 1)], np.int32)        # every pair in every other expert's, descending between
    else:
        q[::3], q[1::3] = -1, P
    plan = mhc.ExpertsPlan(to_dev(o, dev), to_dev(q, dev), (T, k))
    case(f"a plan of any content {kind} T={T} k={k} E={E} D={D} F={F}")
    x, gate = randn(T, D), mhc.mhc_mxfp4(randn(E, F, D))
    full = torch.full((T + 2, k, F), 7.0, dtype=torch.bfloat16, device=dev)
    mhc.mhc_experts_glu(x, plan, gate, gate, out=full[1:T + 1])
    torch.cuda.synchronize()
    assert (full[0] == 7).all() and (full[T + 1] == 7).all()
    # back: [T k, D] to F columns, as the gated projection's rows
    h, down, ones = randn(T, k, D), mhc.mhc_mxfp4(randn(E, F, D)), torch.ones(T, k, device=dev)
    for short in (False, True):
        back = torch.full((T + 2, F), 7.0, dtype=torch.bfloat16, device=dev)
        mhc.mhc_experts_down(h, plan, ones, down, short_terms=short, out=back[1:T + 1])
        torch.cuda.synchronize()
        assert (back[0] == 7).all() and (back[T + 1] == 7).all()
    if kind == 3:
        good = mhc.mhc_experts_glu(x, plan._replace(pairs=to_dev(np.arange(P, dtype=np.int32), dev)), gate, gate)
        named = torch.zeros(P, dtype=torch.bool, device=dev)
        named[2::3] = True
        flat = full[1:T + 1].reshape(P, F)
        assert torch.equal(flat[named], good.reshape(P, F)[named]) and (flat[~named] == 7).all()


@pytest.mark.parametrize("T,k,E,D,F,shape", FAR)
def test_weights_past_32_bits(T, k, E, D, F, shape):
    # the last expert's codes lie past 2^32 bytes; exact sums, multiples of 1/4 up to 36 times the reduction
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    case(f"experts past 32 bits T={T} E={E} D={D} F={F}")
    gen = torch.Generator(device=dev).manual_seed(3)
    some = lambda *s: torch.randint(0, 256, s, generator=gen, device=dev, dtype=torch.uint8)
    scales = lambda *s: torch.full((*s[:-1], s[-1] // 32), 127, dtype=torch.uint8, device=dev)
    e = np.full((T, k), E - 1, np.int32)
    e[:, 1] = 0
    p, p1 = a_plan(e, E, dev), a_plan(np.stack([np.zeros(T), np.full(T, -1)], 1).astype(np.int32), 1, dev)

    def weights(rows, width):
        one = mhc.Mxfp4(some(1, rows, width // 2), scales(1, rows, width), torch.bfloat16, width)
        codes = torch.zeros((E, rows, width // 2), dtype=torch.uint8, device=dev)
        assert (E - 1) * rows * (width // 2) >= 1 << 32
        codes[E - 1] = one.codes[0]
        return mhc.Mxfp4(codes, scales(E, rows, width), torch.bfloat16, width), one

    w, one = weights(F, D)
    x = mhc.Mxfp4(some(T, D // 2), scales(T, D), torch.bfloat16, D)
    h, h1 = mhc.mhc_experts_glu(x, p, w, w), mhc.mhc_experts_glu(x, p1, one, one)
    assert torch.equal(h[:, 0], h1[:, 0]) and (h[:, 1] == 0).all() and (h1[:, 0] != 0).any()
    del w, one, h, h1
    w, one = weights(D, F)
    h = mhc.Mxfp4(some(T, k, F // 2), scales(T, k, F), torch.bfloat16, F)
    wt = torch.ones(T, k, device=dev)
    y, y1 = mhc.mhc_experts_down(h, p, wt, w), mhc.mhc_experts_down(h, p1, wt, one)
    assert torch.equal(y, y1) and (y != 0).any()


@pytest.mark.parametrize("T,k,E,D,F,shape", FAR_RESULTS)
def test_results_past_32_bits(T, k, E, D, F, shape):
    # the last tokens' terms wait for their sum past 2^32 bytes
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    case(f"results past 32 bits T={T} E={E} D={D} F={F}")
    rng = np.random.default_rng(T)
    assert (T - 100) * k * D * 2 >= 1 << 32
    for f16, short in FORMS:
        w = to_mxfp4(*mxfp4(rng, E, D, F, low=127, high=128), F, f16, dev)
        h = to_mxfp4(*mxfp4(rng, T, k, F, low=127, high=128), F, f16, dev)
        e = rng.integers(0, E, (T, k)).astype(np.int32)
        wt = torch.ones(T, k, device=dev)
        y = mhc.mhc_experts_down(h, a_plan(e, E, dev), wt, w, short_terms=short)
        for rows in (slice(0, 100), slice(T - 100, T)):
            few = h._replace(codes=h.codes[rows].contiguous(), scales=h.scales[rows].contiguous())
            v = mhc.mhc_experts_down(few, a_plan(e[rows], E, dev), wt[rows], w)
            if f16 or not short:
                assert torch.equal(y[rows], v)
            else:   # multiples of 1/4 under 2^12: terms in 11 bits and the few tokens' in fp32 differ by 2^-11 of them, and each is rounded once
                near = v.double().abs() * (2.0 ** -11 + 2 * 2.0 ** -8) + 2.0 ** -39 * 4096
                assert ((y[rows].double() - v.double()).abs() <= near).all()
        del w, h, y
