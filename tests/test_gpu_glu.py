"""The gated projection and its backward on the GPU against the formulas in 64 bits.

Tolerances, with e = eps / 2 of the 16-bit format (2^-8 bf16, 2^-11 fp16) and u = 2^-24. A product of two 16-bit values is
exact in fp32, and a sum of K of them, in whatever grouping, is off by at most K u A (A the sum of |terms|); the matrix
cores add in groups, so that bound is wide. |act| has slope at most 1.13 and |act'| at most 1.13; act' itself at most 1.13 in
magnitude and of slope at most 0.8 (GELU's tanh form: both within these to its second digit). So with
eg = D u Ag, eu = D u Au the errors of g and u, and 2^-21 relative for the exponential, the reciprocal and the products:
  h         1.13 eg |u| + |a| eu + 2^-21 |a u|, then one rounding
  dg, du    |dh| (1.13 eu + 0.8 eg |u|) + 2^-21 |dh u| and |dh| 1.13 eg + 2^-21 |dh a|, then one rounding, e |dg|
  grad_x    the sum over f of those errors times |W|, plus 2 F u A, then one rounding
  grad_w    the sum over t of those errors times |x|, plus T u A, then one rounding
A result's rounding is half a step of its value; the first error can move it by as much again."""
import sys

import numpy as np
import pytest

from gpu_helpers import device, to_host
from train_helpers import half_step, load, to_16

pytestmark = pytest.mark.gpu
U, FN = 2.0 ** -24, 2.0 ** -21


def inputs(T, D, F, f16, seed, wide=1.0):
    rng = np.random.default_rng(seed)
    f = lambda *s, std=1.0: to_16(std * rng.standard_normal(s), f16)
    return dict(x=to_16(rng.standard_normal((T, D)) * np.exp(0.5 * rng.standard_normal(D)), f16), w_gate=f(F, D, std=wide / np.sqrt(D)),
                w_up=f(F, D, std=1 / np.sqrt(D)), grad_h=f(T, F))


def act_ref(g, act):
    with np.errstate(over="ignore"):
        if act == "silu":
            s, dz = 1 / (1 + np.exp(-g)), 1.0
        else:
            c, q = 2 * np.sqrt(2 / np.pi), 0.044715
            s, dz = 1 / (1 + np.exp(-c * (g + q * g ** 3))), c * (1 + 3 * q * g * g)
    return g * s, s + g * s * (1 - s) * dz


def reference(x, wg, wu, gh, act, f16):
    """{name: (value, error bound before the rounding)}"""
    e = 2.0 ** -11 if f16 else 2.0 ** -8
    D, (T, F) = x.shape[1], gh.shape
    g, u = x @ wg.T, x @ wu.T
    eg, eu = D * U * (abs(x) @ abs(wg).T), D * U * (abs(x) @ abs(wu).T)
    a, da = act_ref(g, act)
    out = {"h": (a * u, 1.13 * eg * abs(u) + abs(a) * eu + FN * abs(a * u))}
    dg, du = gh * u * da, gh * a
    edg = abs(gh) * (1.13 * eu + 0.8 * eg * abs(u)) + FN * abs(gh * u)
    edu = abs(gh) * 1.13 * eg + FN * abs(gh * a)
    edg, edu = edg + half_step(abs(dg) + edg, f16), edu + half_step(abs(du) + edu, f16)
    out["grad_x"] = (dg @ wg + du @ wu, edg @ abs(wg) + edu @ abs(wu) + 2 * F * U * ((abs(dg) + edg) @ abs(wg) + (abs(du) + edu) @ abs(wu)))
    out["grad_w_gate"] = (dg.T @ x, edg.T @ abs(x) + T * U * ((abs(dg) + edg).T @ abs(x)))
    out["grad_w_up"] = (du.T @ x, edu.T @ abs(x) + T * U * ((abs(du) + edu).T @ abs(x)))
    return out


def check(name, got, ref, f16):
    want, lim = ref
    lim = lim + half_step(np.abs(want) + lim, f16)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= lim).all(), (name, float(np.nanmax(err / lim)), int((~(err <= lim)).sum()), np.argwhere(~(err <= lim))[:4].tolist())
    return float((err / lim).max())


SIZES = [(1, 8, 8), (1, 264, 1000), (2, 40, 24), (7, 1000, 72), (16, 512, 136), (17, 96, 2048), (33, 2056, 264), (64, 128, 1032), (65, 72, 40),
         (127, 1032, 200), (128, 64, 64), (129, 256, 128), (257, 520, 1096), (300, 2048, 544), (1000, 136, 72), (520, 4104, 40), (40, 8, 4104),
         (2049, 48, 56)]


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("T,D,F", SIZES)
def test_forward_and_backward(T, D, F, f16, act):
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    i = inputs(T, D, F, f16, seed=T + D + F, wide=2.0)
    d = {k: v.to(dev) for k, v in i.items()}
    v = {k: t.double().numpy() for k, t in i.items()}
    dt = d["x"].dtype
    print(f"[case] glu T={T} D={D} F={F} f16={f16} {act}", file=sys.stderr, flush=True)
    ref = reference(v["x"], v["w_gate"], v["w_up"], v["grad_h"], act, f16)
    full = torch.full((T + 1, F), 7.0, dtype=dt, device=dev)      # the row behind the last token stays as it was
    h = mhc.mhc_glu(d["x"], d["w_gate"], d["w_up"], act=act, out=full[:T])
    check("h", h, ref["h"], f16)
    assert (full[T] == 7.0).all()
    for kept in (False, True):
        print(f"[case] glu_backward T={T} D={D} F={F} f16={f16} {act} kept={kept}", file=sys.stderr, flush=True)
        x = mhc.mhc_checkpoint(d["x"]) if kept else d["x"]
        if kept:
            ref = reference(load(to_host(x.codes), to_host(x.scales)), v["w_gate"], v["w_up"], v["grad_h"], act, f16)
        rows = dict(grad_x=(T, D), grad_w_gate=(F, D), grad_w_up=(F, D), h=(T, F))
        guard = {k: torch.full((r + 1, c), 7.0, dtype=dt, device=dev) for k, (r, c) in rows.items()}
        got = mhc.mhc_glu_backward(d["grad_h"], x, d["w_gate"], d["w_up"], act=act, need_h=True, out={k: g[:-1] for k, g in guard.items()})
        for k, t in got.items():
            check(k, t, ref[k], f16)
        assert all((g[-1] == 7.0).all() for g in guard.values())
        if not kept:
            assert torch.equal(got["h"], h) or T <= 64   # one kernel computes both (few tokens: another one the forward)
        again = mhc.mhc_glu_backward(d["grad_h"], x, d["w_gate"], d["w_up"], act=act)
        assert set(again) == {"grad_x", "grad_w_gate", "grad_w_up"}
        assert all(torch.equal(again[k], got[k]) for k in again)


@pytest.mark.parametrize("T,D,F", [(4096, 1024, 2048), (1030, 2560, 4104)])
def test_many_tiles_against_float32(T, D, F):
    # sizes of many tiles: whole rows of each result against 64 bits, on the GPU
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    print(f"[case] glu many tiles T={T} D={D} F={F}", file=sys.stderr, flush=True)
    d = {k: v.to(dev) for k, v in inputs(T, D, F, False, seed=1).items()}
    h = mhc.mhc_glu(d["x"], d["w_gate"], d["w_up"])
    got = mhc.mhc_glu_backward(d["grad_h"], d["x"], d["w_gate"], d["w_up"], need_h=True)
    assert torch.equal(got["h"], h)
    x, wg, wu, gh = (d[k].double() for k in ("x", "w_gate", "w_up", "grad_h"))
    g, u = x @ wg.t(), x @ wu.t()
    s = torch.sigmoid(g)
    dg, du = gh * u * (s + g * s * (1 - s)), gh * g * s
    e = 2.0 ** -8
    for name, out, want, mag in (("h", h, g * s * u, None), ("grad_x", got["grad_x"], dg @ wg + du @ wu, dg.abs() @ wg.abs() + du.abs() @ wu.abs()),
                                 ("grad_w_gate", got["grad_w_gate"], dg.t() @ x, dg.abs().t() @ x.abs()),
                                 ("grad_w_up", got["grad_w_up"], du.t() @ x, du.abs().t() @ x.abs())):
        # one rounding of the result and of each of dg and du (e A), and fp32 sums of g and u (2^-12 covers D u Ag with
        # Ag < 16 for these inputs), of the result (65536 u A < 2^-8 A)
        lim = e * want.abs() + 2.0 ** -12 * (1 + (u.abs().max() if mag is None else 0)) if mag is None else e * want.abs() + 2 * e * mag
        assert ((out.double() - want).abs() <= lim).all(), name


def test_against_differences():
    # the directional derivative of L = sum(grad_h h(x, Wg, Wu)), by central differences of the formula in 64 bits at the
    # same inputs: a step of 1e-4 leaves an error of 1e-8 of third derivatives, far below the 16-bit gradients'
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    for act in ("silu", "gelu_tanh"):
        print(f"[case] glu differences {act}", file=sys.stderr, flush=True)
        i = inputs(70, 200, 152, True, seed=9, wide=2.0)
        got = mhc.mhc_glu_backward(*(i[k].to(dev) for k in ("grad_h", "x", "w_gate", "w_up")), act=act)
        v = {k: t.double().numpy() for k, t in i.items()}
        rng = np.random.default_rng(2)

        def loss(x, wg, wu):
            return (v["grad_h"] * act_ref(x @ wg.T, act)[0] * (x @ wu.T)).sum()

        for n, (name, grad) in enumerate((("x", "grad_x"), ("w_gate", "grad_w_gate"), ("w_up", "grad_w_up"))):
            step = rng.standard_normal(v[name].shape)
            at = lambda s: loss(*[v[k] + (s * step if k == name else 0) for k in ("x", "w_gate", "w_up")])
            diff = (at(1e-4) - at(-1e-4)) / 2e-4
            g = got[grad].double().cpu().numpy()
            # the gradients' roundings (2^-11 each, twice), of random sign against the step's: 8 standard deviations
            lim = 8 * 2.0 ** -10 * np.sqrt(((g * step) ** 2).sum()) + 1e-6 * np.abs(g * step).sum()
            assert abs((g * step).sum() - diff) <= lim, (act, name, (g * step).sum(), diff, lim)


def test_values_that_are_not_finite_stay_in_their_token():
    # NaN and infinities in one token's x and grad_h, at the ends of the rows where a tile's reduction stops short of a stage
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    for T, D, F in ((40, 72, 40), (130, 264, 136), (300, 40, 72)):
        print(f"[case] glu not finite T={T} D={D} F={F}", file=sys.stderr, flush=True)
        d = {k: v.to(dev) for k, v in inputs(T, D, F, False, seed=4).items()}
        clean = mhc.mhc_glu(d["x"], d["w_gate"], d["w_up"])
        base = mhc.mhc_glu_backward(d["grad_h"], d["x"], d["w_gate"], d["w_up"])
        t = T // 2
        d["x"][t, 0] = float("nan")
        d["grad_h"][t, 0], d["grad_h"][t, -1] = float("inf"), float("nan")
        keep = [k for k in range(T) if k != t]
        h = mhc.mhc_glu(d["x"], d["w_gate"], d["w_up"])
        assert torch.equal(h[keep], clean[keep]) and torch.isnan(h[t]).all()
        got = mhc.mhc_glu_backward(d["grad_h"], d["x"], d["w_gate"], d["w_up"])
        assert torch.equal(got["grad_x"][keep], base["grad_x"][keep]) and torch.isnan(got["grad_x"][t]).all()


def test_extreme_gates():
    # gates far out: act(g) is g or 0 there and act'(g) 1 or 0, with nothing left of the cube's overflow
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    print("[case] glu extreme gates", file=sys.stderr, flush=True)
    size = torch.tensor([3e1, -3e1, 1e4, -1e4, 1e15, -1e15, 3e38, -3e38], dtype=torch.bfloat16)
    x = torch.zeros((8, 8), dtype=torch.bfloat16)
    x[:, 0], x[:, 1] = size, 1.0
    w = torch.zeros((8, 8), dtype=torch.bfloat16)
    w[:, 0] = 1.0
    wu = torch.zeros((8, 8), dtype=torch.bfloat16)
    wu[:, 1] = 1.0
    gh = torch.ones((8, 8), dtype=torch.bfloat16)
    x, w, wu, gh = (t.to(dev) for t in (x, w, wu, gh))
    for act in ("silu", "gelu_tanh"):
        h = mhc.mhc_glu(x, w, wu, act=act).float().cpu()
        want = torch.where(size > 0, size, torch.zeros_like(size)).float()
        assert ((h - want[:, None]).abs() <= 2e-10 * size.abs().float()[:, None] + 1e-9).all()
        got = mhc.mhc_glu_backward(gh, x, w, wu, act=act)
        # grad_x[:, 0] = sum_f act'(g) = 8 or 0
        gx = got["grad_x"].float().cpu()[:, 0]
        assert ((gx - torch.where(size > 0, 8.0, 0.0)).abs() <= 1e-6).all(), (act, gx)


def test_empty_and_leading_dimensions():
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    print("[case] glu empty", file=sys.stderr, flush=True)
    w = torch.ones((72, 40), dtype=torch.float16, device=dev)
    x = torch.empty((0, 40), dtype=torch.float16, device=dev)
    assert mhc.mhc_glu(x, w, w).shape == (0, 72)
    for kept in (x, mhc.mhc_checkpoint(x)):
        out = {k: torch.full(s, 7.0, dtype=torch.float16, device=dev) for k, s in (("grad_x", (0, 40)), ("grad_w_gate", (72, 40)), ("grad_w_up", (72, 40)))}
        mhc.mhc_glu_backward(torch.empty((0, 72), dtype=torch.float16, device=dev), kept, w, w, out=out)
        assert not out["grad_w_gate"].any() and not out["grad_w_up"].any()
    d = {k: v.to(dev) for k, v in inputs(30, 40, 72, True, seed=4).items()}
    h = mhc.mhc_glu(d["x"].reshape(2, 15, 40), d["w_gate"], d["w_up"])
    assert h.shape == (2, 15, 72) and torch.equal(h.reshape(30, 72), mhc.mhc_glu(d["x"], d["w_gate"], d["w_up"]))
    got = mhc.mhc_glu_backward(d["grad_h"].reshape(2, 15, 72), mhc.mhc_checkpoint(d["x"].reshape(2, 15, 40)), d["w_gate"], d["w_up"], need_h=True)
    assert got["grad_x"].shape == (2, 15, 40) and got["h"].shape == (2, 15, 72)
