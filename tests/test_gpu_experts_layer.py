"""The experts' operators run together, as a program uses them: serving between mhc_pre and mhc_post with padded tokens,
captured into HIP graphs and on two streams at once; training with the gated projection of 16-bit weights for each expert."""
import sys

import numpy as np
import pytest

import synth
import test_gpu_experts as products
from experts_helpers import U, act_ref, check, half_step, mxfp4, plan, rounded, route, sum_error, to_16, to_mxfp4, values
from gpu_helpers import device, to_dev

pytestmark = pytest.mark.gpu


def part_error(v):
    """Rounding the pairs' results [P, D] to 11 bits under the power of two of 32 of them, at most."""
    P, D = v.shape
    b = np.pad(np.abs(v), ((0, 0), (0, -D % 32))).reshape(P, -1, 32).max(-1)
    return 2.0 ** -11 * np.abs(v) + 2.0 ** -39 * np.repeat(b, 32, -1)[:, :D]


class Layer:
    """streams -> pre -> h_in -> router -> experts -> post -> streams; tokens past `real` are padding."""
    E, k, n = 24, 4, 4
    rules = dict(score="sigmoid", groups=4, top_groups=2, scale=2.5)

    def __init__(self, T, D, F, f16, seed, real=None):
        import torch
        self.torch, self.dev, self.T, self.D, self.F, self.f16 = torch, device(), T, D, F, f16
        self.real = T if real is None else real
        rng = np.random.default_rng(seed)
        inp = synth.custom(T, self.n, D, gamma=False, need_backward=False, num_iters=20, seed=seed, x_f16=f16)
        self.x, self.phi, self.alpha, self.bias = (to_dev(a, self.dev, f16) for a in (inp.x, inp.phi, inp.alpha, inp.bias))
        self.router = torch.from_numpy((rng.standard_normal((self.E, D)) / np.sqrt(D)).astype(np.float32)).to(self.dev)
        self.balance = torch.from_numpy((0.05 * rng.standard_normal(self.E)).astype(np.float32)).to(self.dev)
        E = self.E
        self.wg, self.wu, self.wd = mxfp4(rng, E, F, D, low=121, high=125), mxfp4(rng, E, F, D, low=121, high=125), mxfp4(rng, E, D, F, low=121, high=125)
        self.gate, self.up, self.down = (to_mxfp4(*w, s, f16, self.dev) for w, s in ((self.wg, D), (self.wu, D), (self.wd, F)))

    def __call__(self, x=None):
        import mhc_hyper_connection_amd as mhc
        r = {}
        x = self.x if x is None else x
        r["h_in"], h_post, h_res = mhc.mhc_pre(x, self.phi, self.alpha, self.bias)[:3]
        r["logits"] = (r["h_in"].float()[:, None, :] * self.router).sum(-1)
        r["logits"][self.real:] = -np.inf
        r["weights"], r["experts"] = mhc.mhc_route(r["logits"], self.k, bias=self.balance, **self.rules)
        p = mhc.mhc_experts_plan(r["experts"], self.E)
        r["offsets"], r["pairs"] = p.offsets, p.pairs
        r["h"] = mhc.mhc_experts_glu(r["h_in"], p, self.gate, self.up)
        r["y"] = mhc.mhc_experts_down(r["h"], p, r["weights"], self.down)
        r["h_post"], r["h_res"] = h_post, h_res
        r["out"] = mhc.mhc_post(r["y"], x, h_post, h_res)
        return r


@pytest.mark.parametrize("T,D,F,f16,real", [(1, 264, 520, False, 1), (9, 256, 136, True, 7), (130, 264, 200, False, 97), (700, 128, 264, True, 700),
                                            (1500, 96, 136, False, 1403), (33, 520, 72, False, 0)])
def test_serving(T, D, F, f16, real):
    import torch
    print(f"[case] experts' layer T={T} D={D} F={F} f16={f16} real={real}", file=sys.stderr, flush=True)
    L = Layer(T, D, F, f16, seed=T, real=real)
    got = L()
    torch.cuda.synchronize()
    host = {a: b.double().cpu().numpy() if b.is_floating_point() else b.cpu().numpy() for a, b in got.items()}
    # each step in 64 bits from what the one before gave
    w, e = route(host["logits"], L.k, L.balance.double().cpu().numpy(), **L.rules)
    assert np.array_equal(host["experts"], e) and (e[real:] == -1).all() and (real == 0 or (e[:real] >= 0).all())
    assert (np.abs(host["weights"] - w) <= np.maximum(U * np.abs(w), 2.0 ** -150) * (1 + 2.0 ** -16)).all()
    offsets, pairs = plan(e, L.E)
    assert np.array_equal(host["offsets"], offsets) and np.array_equal(host["pairs"], pairs)
    flat, tok = e.reshape(-1), np.arange(T * L.k) // L.k
    xv, hv = rounded(host["h_in"], f16), rounded(host["h"], f16).reshape(T * L.k, F)
    gv, uv, dv = values(*L.wg, D), values(*L.wu, D), values(*L.wd, F)
    g, u, ag, au = (np.zeros((T * L.k, F)) for _ in range(4))
    y, ay = np.zeros((T * L.k, D)), np.zeros((T * L.k, D))
    for i in np.unique(flat[flat >= 0]):
        at = flat == i
        x = xv[tok[at]]
        g[at], u[at], ag[at], au[at] = x @ gv[i].T, x @ uv[i].T, np.abs(x) @ np.abs(gv[i]).T, np.abs(x) @ np.abs(uv[i]).T
        y[at], ay[at] = hv[at] @ dv[i].T, np.abs(hv[at]) @ np.abs(dv[i]).T
    a = act_ref(g, "silu")
    check("h", got["h"].reshape(T * L.k, F), a * u, 1.13 * sum_error(D, ag) * np.abs(u) + np.abs(a) * sum_error(D, au) + 2.0 ** -21 * np.abs(a * u), f16)
    err = sum_error(F, ay)
    if not f16:
        err = err + part_error(np.abs(y) + err)
    wt = np.abs(host["weights"]).reshape(-1, 1)
    lim = (wt * err).reshape(T, L.k, D).sum(1) + (L.k + 1) * U * (wt * np.abs(y)).reshape(T, L.k, D).sum(1)
    check("y", got["y"], (host["weights"].reshape(-1, 1) * y).reshape(T, L.k, D).sum(1), lim, f16)
    assert (host["y"][real:] == 0).all()
    # post: 5 products of fp32 and 16-bit values, fused: 2^-20 of the terms, and its rounding
    x = L.x.double().cpu().numpy()
    terms = [host["h_post"][:, :, None] * host["y"][:, None, :]] + [host["h_res"][:, i, :, None] * x[:, i, None, :] for i in range(L.n)]
    check("out", got["out"], sum(terms), 2.0 ** -20 * sum(np.abs(t) for t in terms), f16)


@pytest.mark.parametrize("T", [2, 150, 1100])
def test_captured_into_graphs(T):
    import torch
    print(f"[case] experts' layer in graphs T={T}", file=sys.stderr, flush=True)
    L = Layer(T, 264, 200, False, seed=5, real=T - T // 10)
    xs = [L.x.clone(), L.x.roll(1, 0) * 0.5, -L.x]
    want = [{a: b.clone() for a, b in L(x).items()} for x in xs]
    x = L.x.clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream(L.dev)
    side.wait_stream(torch.cuda.current_stream(L.dev))
    with torch.cuda.stream(side):
        L(x)
    torch.cuda.current_stream(L.dev).wait_stream(side)
    torch.cuda.synchronize()
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        a = L(x)
    with torch.cuda.graph(second):        # a second graph, with workspaces of its own
        b = L(x)
    for rep in range(6):
        for v in (*a.values(), *b.values()):
            v.view(torch.uint8).fill_(0x7F)
        x.copy_(xs[rep % 3])              # the replays' routing changes with their input
        eager = L(xs[(rep + 1) % 3])
        first.replay()
        if rep % 2:
            torch.cuda.synchronize()
        second.replay()
        torch.cuda.synchronize()
        for name, w in want[rep % 3].items():
            for r in (a, b):
                assert torch.equal(r[name].view(torch.uint8), w.view(torch.uint8)), (rep, name)
            assert torch.equal(eager[name].view(torch.uint8), want[(rep + 1) % 3][name].view(torch.uint8)), (rep, name)


def test_on_two_streams_at_once():
    import torch
    layers = [Layer(300, 264, 200, False, seed=11), Layer(2, 136, 520, True, seed=12)]
    want = [{a: b.clone() for a, b in L().items()} for L in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(layers[0].dev) for _ in layers]
    got = [[], []]
    for rep in range(8):
        for i, (L, s) in enumerate(zip(layers, streams)):
            with torch.cuda.stream(s):
                got[i].append(L())
    torch.cuda.synchronize()
    for rs, w in zip(got, want):
        for r in rs:
            for name in w:
                assert torch.equal(r[name].view(torch.uint8), w[name].view(torch.uint8)), name


@pytest.mark.parametrize("f16,score,renormalise", [(False, "softmax", True), (True, "sigmoid", True), (False, "softmax", False)])
def test_training_step(f16, score, renormalise):
    """The experts trained in 16 bits: mhc_route and its plan, mhc_glu of each expert's rows, and the way back."""
    import mhc_hyper_connection_amd as mhc
    import torch
    print(f"[case] experts' training f16={f16} {score} renormalise={renormalise}", file=sys.stderr, flush=True)
    T, E, k, D, F, dev = 150, 6, 2, 136, 264, device()
    rng = np.random.default_rng(7)
    t = lambda *s, std=1.0: to_16(std * rng.standard_normal(s), f16).to(dev)
    x, wg, wu, wd = t(T, D), t(E, F, D, std=2 / np.sqrt(D)), t(E, F, D, std=1 / np.sqrt(D)), t(E, D, F, std=1 / np.sqrt(F))
    gy = t(T, D)
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(dev)
    rule = dict(score=score, renormalise=renormalise)
    w, e = mhc.mhc_route(logits, k, **rule)
    p = mhc.mhc_experts_plan(e, E)
    off = p.offsets.tolist()
    h = torch.zeros(T * k, F, dtype=x.dtype, device=dev)
    rows = [p.pairs[off[i]:off[i + 1]].long() for i in range(E)]
    for i, r in enumerate(rows):
        h[r] = mhc.mhc_glu(x[r // k], wg[i], wu[i])
    grad_w, grad_x, grad_gate, grad_up = torch.zeros(T * k, device=dev), torch.zeros(T, D, device=dev), [], []
    for i, r in enumerate(rows):
        back = gy[r // k].float() @ wd[i].float()                        # the gradient of h, but for the weight
        grad_w[r] = (back * h[r].float()).sum(1)
        g = mhc.mhc_glu_backward((w.reshape(-1)[r, None] * back).to(x.dtype), x[r // k], wg[i], wu[i])
        grad_x.index_put_((r // k,), g["grad_x"].float(), accumulate=True)
        grad_gate.append(g["grad_w_gate"])
        grad_up.append(g["grad_w_up"])
    grad_logits = mhc.mhc_route_backward(grad_w.reshape(T, k), logits, w, e, **rule)
    # by differentiation in 64 bits
    d = lambda v: v.double().cpu().requires_grad_()
    x8, wg8, wu8, l8 = d(x), d(wg), d(wu), d(logits)
    s = torch.softmax(l8, -1) if score == "softmax" else torch.sigmoid(l8)
    c = s.gather(1, e.long().cpu())
    c = c / c.sum(1, keepdim=True) if renormalise else c
    y = torch.zeros(T, D, dtype=torch.float64)
    for i in range(E):
        for j in range(k):
            at = (e[:, j] == i).cpu().nonzero()[:, 0]
            g = x8[at] @ wg8[i].t()
            y = y.index_add(0, at, c[at, j, None] * ((g * torch.sigmoid(g) * (x8[at] @ wu8[i].t())) @ wd[i].double().cpu().t()))
    (y * gy.double().cpu()).sum().backward()
    # On the way to a gradient are at most 5 roundings to 16 bits (h, the gradient of h, dg and du, the result), each at most
    # eps / 2 of its tensor's norm, and none of the maps in between (projections of about unit gain, an activation of slope
    # at most 1.13, the weights' differences) carries a relative error on by more than 4; a wrong term is of order 1.
    lim = 20 * torch.finfo(x.dtype).eps / 2
    rel = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())
    for name, a, b in (("logits", grad_logits, l8.grad), ("x", grad_x, x8.grad), ("gate", torch.stack(grad_gate), wg8.grad), ("up", torch.stack(grad_up), wu8.grad)):
        assert rel(a, b) <= lim, (name, rel(a, b), lim)


def test_the_forms_in_16_and_in_4_bits_agree():
    """x, h and weights that 4 bits hold exactly: the experts' products against the gated projection and the plain
    product in 16 bits, each within its own rounding of h."""
    import mhc_hyper_connection_amd as mhc
    import torch
    T, E, k, D, F, dev = 70, 5, 2, 128, 96, device()
    rng = np.random.default_rng(3)
    x4, gate, up = (to_mxfp4(*mxfp4(rng, *s, low=a, high=b), D, False, dev) for s, a, b in (((T, D), 126, 128), ((E, F, D), 121, 124), ((E, F, D), 121, 124)))
    x, wg, wu = (mhc.mhc_mxfp4_restore(m) for m in (x4, gate, up))
    e = torch.from_numpy(np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)).to(dev)
    p = mhc.mhc_experts_plan(e, E)
    h = mhc.mhc_experts_glu(x, p, gate, up).reshape(T * k, F)
    assert torch.equal(h, mhc.mhc_experts_glu(x4, p, gate, up).reshape(T * k, F))
    off = p.offsets.tolist()
    for i in range(E):
        r = p.pairs[off[i]:off[i + 1]].long()
        a, b = h[r].double().cpu().numpy(), mhc.mhc_glu(x[r // k], wg[i], wu[i]).double().cpu().numpy()
        xr, g, u = (v.double().cpu().numpy() for v in (x[r // k], wg[i], wu[i]))
        gs, us = xr @ g.T, xr @ u.T
        act = np.abs(act_ref(gs, "silu"))
        lim = 1.13 * sum_error(D, np.abs(xr) @ np.abs(g).T) * np.abs(us) + act * sum_error(D, np.abs(xr) @ np.abs(u).T) + 2.0 ** -21 * act * np.abs(us)
        assert (np.abs(a - b) <= 2 * (lim + half_step(act * np.abs(us) + lim, False))).all()


@pytest.mark.parametrize("T,k,E,D,F,f16", [(20000, 1, 150, 1288, 264, False), (40000, 1, 3, 1032, 264, True), (30000, 1, 2, 1024, 264, False),
                                           (6000, 4, 90, 256, 520, True)])
def test_workgroups_that_take_several_units(T, k, E, D, F, f16):
    # more units than places for workgroups, small tiles and large, reductions that end inside a group of stages and with one
    products.test_experts(T, k, E, D, F, f16)


@pytest.mark.parametrize("T,K,N", [(9000, 1032, 4104), (20000, 2048, 1032)])
def test_a_product_of_several_units(T, K, N):
    products.test_product(T, K, N, False)
