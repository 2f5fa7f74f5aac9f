"""hc_post's backward on the GPU against its formulas in 64 bits, from 16-bit activations and from 8-bit checkpoints.

Tolerances, with u = 2^-24 and A the sum of |terms|:
  grad_x, grad_residual (16 bits): n terms in a chain of fused multiply-adds, an error of at most n u A, then one rounding
      (half a step of the result, whose size the first error may change: another n u A covers it).
  grad_post, grad_comb (f32): a lane adds ceil(D/8 / lanes) octets one value after another, then 6 levels join 64 lanes and
      2 four waves. (L + 8) u A bounds it with L = 8 ceil(D/8 / 64) values in a lane (a quarter with four waves)."""
import sys

import numpy as np
import pytest

from gpu_helpers import device, to_host
from train_helpers import half_step, load, to_16

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def inputs(T, n, D, f16, seed):
    rng = np.random.default_rng(seed)
    size = np.exp(rng.standard_normal(D))
    f = lambda *s: to_16(rng.standard_normal(s), f16)
    return dict(grad_out=f(T, n, D), x=to_16(rng.standard_normal((T, D)) * size, f16), residual=to_16(rng.standard_normal((T, n, D)) * size, f16),
                post=rng.uniform(0, 2, (T, n)).astype(np.float32), comb=rng.standard_normal((T, n, n)).astype(np.float32))


def reference(go, x, r, post, comb):
    """(value, sum of |terms|) of each gradient."""
    out = {}
    for k, f in (("v", lambda a: a), ("a", np.abs)):
        g, xx, rr, p, c = f(go), f(x), f(r), f(post.astype(np.float64)), f(comb.astype(np.float64))
        out[k] = dict(grad_x=np.einsum("tj,tjd->td", p, g), grad_residual=np.einsum("tij,tjd->tid", c, g),
                      grad_post=np.einsum("tjd,td->tj", g, xx), grad_comb=np.einsum("tid,tjd->tij", rr, g))
    return out["v"], out["a"]


def check(got, go, x, r, post, comb, f16):
    n, D = go.shape[1:]
    want, mag = reference(go, x, r, post, comb)
    L = 8 * -(-D // 512)
    for k, v in got.items():
        lim = (half_step(want[k], f16) + 2 * n * U * mag[k]) if k in ("grad_x", "grad_residual") else (L + 8) * U * mag[k] + 1e-38
        err = np.abs(v.double().cpu().numpy() - want[k])
        assert (err <= lim).all(), (k, float((err / lim).max()))


CASES = [(1, 4, 8), (3, 4, 40), (2, 6, 1000), (65, 8, 520), (130, 4, 2048), (7, 6, 16384), (5, 8, 16384), (4096, 4, 72), (4099, 6, 136),
         (5001, 8, 64), (4097, 4, 1032), (600, 4, 2056), (513, 8, 4104)]


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("T,n,D", CASES)
def test_gradients(T, n, D, f16):
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    i = inputs(T, n, D, f16, seed=T + n + D)
    d = {k: (torch.from_numpy(v) if isinstance(v, np.ndarray) else v).to(dev) for k, v in i.items()}
    go = i["grad_out"].double().numpy()
    for kept in ((), ("x",), ("residual",), ("x", "residual")):
        print(f"[case] post_backward T={T} n={n} D={D} f16={f16} kept={kept}", file=sys.stderr, flush=True)
        acts = {k: mhc.mhc_checkpoint(d[k]) if k in kept else d[k] for k in ("x", "residual")}
        vals = {k: load(to_host(a.codes), to_host(a.scales)) if k in kept else i[k].double().numpy() for k, a in acts.items()}
        # one row more than the gradients have: rows behind the last token stay as they were
        full = dict(grad_x=torch.full((T + 1, D), 7.0, dtype=d["x"].dtype, device=dev), grad_residual=torch.full((T + 1, n, D), 7.0, dtype=d["x"].dtype, device=dev),
                    grad_post=torch.full((T + 1, n), 7.0, device=dev), grad_comb=torch.full((T + 1, n, n), 7.0, device=dev))
        got = mhc.mhc_post_backward(d["grad_out"], acts["x"], acts["residual"], d["post"], d["comb"], out={k: v[:T] for k, v in full.items()})
        check(got, go, vals["x"], vals["residual"], i["post"], i["comb"], f16)
        assert all((v[T] == 7.0).all() for v in full.values())
        again = mhc.mhc_post_backward(d["grad_out"], acts["x"], acts["residual"], d["post"], d["comb"])
        assert all(torch.equal(got[k], again[k]) for k in got)


def test_against_differences():
    # L = <grad_out, post(x, r, post, comb)> is linear in each argument: its change under a step along one argument is the
    # gradient's product with that step, up to mhc_post's rounding of each output (2^-9 of it, of random sign)
    import torch
    import mhc_hyper_connection_amd as mhc
    dev = device()
    T, n, D = 33, 4, 264
    print("[case] post_backward differences", file=sys.stderr, flush=True)
    i = inputs(T, n, D, True, 5)
    d = {k: (torch.from_numpy(v) if isinstance(v, np.ndarray) else v).to(dev) for k, v in i.items()}
    got = mhc.mhc_post_backward(d["grad_out"], d["x"], d["residual"], d["post"], d["comb"])
    rng = np.random.default_rng(1)
    go = d["grad_out"].double()
    for name, grad in (("x", "grad_x"), ("residual", "grad_residual"), ("post", "grad_post"), ("comb", "grad_comb")):
        base = {k: d[k] for k in ("x", "residual", "post", "comb")}
        step = torch.from_numpy(rng.standard_normal(tuple(d[name].shape))).to(d[name].dtype).to(dev)
        up, down = ((d[name].float() + s * step.float()).to(d[name].dtype) for s in (1, -1))
        hi, lo = mhc.mhc_post(**{**base, name: up}).double(), mhc.mhc_post(**{**base, name: down}).double()
        diff = float((go * (hi - lo)).sum())
        want = float((got[grad].double() * (up.double() - down.double())).sum())
        # each output is off by half a step (2^-11 of it); the gradient's elements by 2^-11 too
        lim = float((go.abs() * (hi.abs() + lo.abs())).sum()) * 2.0 ** -11 + float((got[grad].double().abs() * (up.double() - down.double()).abs()).sum()) * 2.0 ** -11
        assert abs(diff - want) <= lim, (name, diff, want, lim)


def test_not_finite_values_stay_where_they_are():
    # an infinity in one token's activations reaches that token's sums and no other token
    import torch
    import mhc_hyper_connection_amd as mhc
    dev = device()
    i = inputs(9, 4, 96, False, 2)
    d = {k: (torch.from_numpy(v) if isinstance(v, np.ndarray) else v).to(dev) for k, v in i.items()}
    print("[case] post_backward not finite", file=sys.stderr, flush=True)
    clean = mhc.mhc_post_backward(d["grad_out"], mhc.mhc_checkpoint(d["x"]), d["residual"], d["post"], d["comb"])
    d["x"][4, 7] = float("inf")
    got = mhc.mhc_post_backward(d["grad_out"], mhc.mhc_checkpoint(d["x"]), d["residual"], d["post"], d["comb"])
    assert torch.isnan(got["grad_post"][4]).all()
    keep = [t for t in range(9) if t != 4]
    assert torch.equal(got["grad_post"][keep], clean["grad_post"][keep])
    for k in ("grad_x", "grad_residual", "grad_comb"):
        assert torch.equal(got[k], clean[k])


def test_empty():
    import torch
    import mhc_hyper_connection_amd as mhc
    dev = device()
    e = torch.empty((0, 6, 64), dtype=torch.bfloat16, device=dev)
    out = mhc.mhc_post_backward(e, e[:, 0], mhc.mhc_checkpoint(e), torch.empty((0, 6), device=dev), torch.empty((0, 6, 6), device=dev))
    assert out["grad_comb"].shape == (0, 6, 6) and out["grad_x"].shape == (0, 64)
