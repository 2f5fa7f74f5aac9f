"""The training operators of a sub-layer run together, as a program uses them: forward with only 8-bit checkpoints kept,
backward from them; captured into a HIP graph; on several streams; over tensors of more than 2^32 values."""
import sys

import numpy as np
import pytest

import synth
from gpu_helpers import device, to_dev
from train_helpers import to_16

pytestmark = pytest.mark.gpu


class SubLayer:
    """streams -> pre -> h_in -> gated projection -> (a plain product) -> post -> streams."""

    def __init__(self, T, n, D, F, f16, seed, iters=20):
        import torch
        self.dev, self.n, self.D, self.iters = device(), n, D, iters
        inp = synth.custom(T, n, D, gamma=True, need_backward=True, num_iters=iters, seed=seed, x_f16=f16)
        self.x, self.phi, self.alpha, self.bias, self.gamma = (to_dev(a, self.dev, f16) for a in (inp.x, inp.phi, inp.alpha, inp.bias, inp.gamma))
        rng = np.random.default_rng(seed)
        f = lambda *s, std=1.0: to_16(std * rng.standard_normal(s), f16).to(self.dev)
        self.wg, self.wu, self.wd = f(F, D, std=2 / np.sqrt(D)), f(F, D, std=1 / np.sqrt(D)), f(D, F, std=1 / np.sqrt(F))
        self.grad_out = f(T, n, D)
        self.torch = torch

    def forward(self):
        import mhc_hyper_connection_amd as mhc
        h_in, h_post, h_res, self.saved = mhc.mhc_pre(self.x, self.phi, self.alpha, self.bias, self.gamma, num_iters=self.iters, need_backward=True)
        self.h_post, self.h_res, self.h_in = h_post, h_res, h_in
        self.h = mhc.mhc_glu(h_in, self.wg, self.wu)
        self.y = (self.h.float() @ self.wd.float().t()).to(h_in.dtype)
        self.out, self.ck_out = mhc.mhc_post_checkpoint(self.y, self.x, h_post, h_res)
        self.kept = {"x": mhc.mhc_checkpoint(self.x), "y": mhc.mhc_checkpoint(self.y), "h_in": mhc.mhc_checkpoint(h_in)}
        return self.out

    def backward(self, x, y, h_in):
        """Gradients from the activations, each a tensor or a Checkpoint."""
        import mhc_hyper_connection_amd as mhc
        s = self.saved
        p = mhc.mhc_post_backward(self.grad_out, y, x, self.h_post, self.h_res)
        grad_h = (p["grad_x"].float() @ self.wd.float()).to(self.x.dtype)
        g = mhc.mhc_glu_backward(grad_h, h_in, self.wg, self.wu, need_h=True)
        q = mhc.mhc_pre_backward(x, self.phi, self.alpha, g["grad_x"], p["grad_post"], p["grad_comb"], s["inv_rms"], s["h_mix"], s["h_pre"],
                                 self.h_post, self.gamma, p["grad_residual"], num_iters=self.iters, sum_out=s["sum_out"], norm_out=s["norm_out"])
        return dict(q, grad_w_gate=g["grad_w_gate"], grad_w_up=g["grad_w_up"], grad_w_down=p["grad_x"].float().t() @ g["h"].float(), h=g["h"])

    def reference(self):
        """The same gradients by differentiation of the whole sub-layer in 64 bits."""
        torch, n, T = self.torch, self.n, self.x.shape[0]
        d = lambda t: t.double().requires_grad_()
        x, phi, alpha, bias, gamma, wg, wu, wd = (d(t) for t in (self.x, self.phi, self.alpha, self.bias, self.gamma, self.wg, self.wu, self.wd))
        xf = x.reshape(T, -1)
        w = (xf * gamma.reshape(-1)) @ phi.t() * torch.rsqrt(xf.square().mean(1, keepdim=True) + 1e-6)
        h_pre = torch.sigmoid(alpha[0] * w[:, :n] + bias[:n]) + 1e-6
        h_post = 2 * torch.sigmoid(alpha[1] * w[:, n:2 * n] + bias[n:2 * n])
        a = torch.softmax((alpha[2] * w[:, 2 * n:] + bias[2 * n:]).reshape(T, n, n), -1) + 1e-6
        for k in range(1, 2 * self.iters):
            a = a / (a.sum(1 if k % 2 else 2, keepdim=True) + 1e-6)
        h_in = (h_pre[:, :, None] * x).sum(1)
        g = h_in @ wg.t()
        y = (g * torch.sigmoid(g) * (h_in @ wu.t())) @ wd.t()
        out = h_post[:, :, None] * y[:, None, :] + torch.einsum("tij,tid->tjd", a, x)
        (out * self.grad_out.double()).sum().backward()
        return dict(grad_x=x.grad, grad_phi=phi.grad, grad_alpha=alpha.grad, grad_bias=bias.grad, grad_gamma=gamma.grad, grad_w_gate=wg.grad,
                    grad_w_up=wu.grad, grad_w_down=wd.grad), out.detach()


@pytest.mark.parametrize("T,n,D,F,f16", [(200, 4, 264, 520, False), (97, 6, 136, 264, True), (130, 8, 96, 200, False)])
def test_training_step(T, n, D, F, f16):
    import mhc_hyper_connection_amd as mhc
    import torch
    print(f"[case] sub-layer T={T} n={n} D={D} F={F} f16={f16}", file=sys.stderr, flush=True)
    L = SubLayer(T, n, D, F, f16, seed=T)
    out = L.forward()
    want, ref_out = L.reference()
    assert torch.equal(L.ck_out.codes, mhc.mhc_checkpoint(out).codes)
    exact = L.backward(L.x, L.y, L.h_in)                 # from the 16-bit activations
    assert torch.equal(exact["h"], L.h) or T <= 64
    # Each gradient's path has at most 10 roundings to 16 bits (h_in, h, y, grad_y, grad_h, dg and du, grad_h_in,
    # grad_residual, the result), each at most e = eps / 2 of its tensor's norm; none of the maps in between (projections
    # of about unit gain, an activation of slope at most 1.13, means over streams) carries a relative error on by
    # more than 4. 40 e bounds the relative error of the norm; a dropped or wrong term is of order 1.
    e = 2.0 ** -11 if f16 else 2.0 ** -8
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())
    assert rel(out, ref_out) <= 40 * e
    for k, v in want.items():
        assert rel(exact[k], v) <= 40 * e, (k, rel(exact[k], v), 40 * e)
    # from the checkpoints alone: the gradients at the values they stand for, bit for bit
    kept = L.backward(L.kept["x"], L.kept["y"], L.kept["h_in"])
    back = {k: mhc.mhc_checkpoint_restore(v) for k, v in L.kept.items()}
    same = L.backward(back["x"], back["y"], back["h_in"])
    for k in kept:
        assert torch.equal(kept[k].view(torch.uint8), same[k].view(torch.uint8)), k
    # an activation is off by at most 1/64 of its block's largest value (half of that but at the top), which for
    # these inputs is within 4 of a value's norm: 1/16 of a tensor's norm, and through the same maps at most 4 times that
    for k, v in want.items():
        assert rel(kept[k], v) <= 40 * e + 0.25, (k, rel(kept[k], v))


@pytest.mark.parametrize("T,D,F", [(300, 264, 520), (20, 136, 264)])
def test_captured_into_a_graph(T, D, F):
    # one token kernel or tiles, cut tiles and their joins: captured once, replayed between eager work of the program
    import mhc_hyper_connection_amd as mhc
    import torch
    print(f"[case] graph T={T} D={D} F={F}", file=sys.stderr, flush=True)
    L = SubLayer(T, 4, D, F, False, seed=3, iters=3)
    L.forward()
    grad_h = to_16(np.random.default_rng(5).standard_normal((T, F)), False).to(L.dev)

    def step():
        s = L.saved
        ck = mhc.mhc_checkpoint(L.h_in)
        p = mhc.mhc_post_backward(L.grad_out, L.kept["y"], L.kept["x"], L.h_post, L.h_res)
        g = mhc.mhc_glu_backward(grad_h, ck, L.wg, L.wu, need_h=True)
        q = mhc.mhc_pre_backward(L.kept["x"], L.phi, L.alpha, g["grad_x"], p["grad_post"], p["grad_comb"], s["inv_rms"], s["h_mix"], s["h_pre"],
                                 L.h_post, L.gamma, p["grad_residual"], num_iters=3, sum_out=s["sum_out"], norm_out=s["norm_out"])
        o, c = mhc.mhc_post_checkpoint(L.y, L.x, L.h_post, L.h_res)
        return {**q, **g, "post": p["grad_comb"], "out": o, "codes": c.codes, "scales": c.scales, "fwd": mhc.mhc_glu(mhc.mhc_checkpoint_restore(ck), L.wg, L.wu)}

    want = {k: v.clone() for k, v in step().items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream(L.dev)
    side.wait_stream(torch.cuda.current_stream(L.dev))
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream(L.dev).wait_stream(side)
    torch.cuda.synchronize()
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        a = step()
    with torch.cuda.graph(second):        # a second graph, with workspaces of its own
        b = step()
    for rep in range(4):
        for v in (*a.values(), *b.values()):
            v.view(torch.uint8).fill_(0x7F)
        eager = step()
        first.replay()
        second.replay()
        torch.cuda.synchronize()
        for k, w in want.items():
            for got in (a, b, eager):
                assert torch.equal(got[k].view(torch.uint8), w.view(torch.uint8)), (rep, k)


def test_calls_on_several_streams():
    import mhc_hyper_connection_amd as mhc
    import torch
    print("[case] streams", file=sys.stderr, flush=True)
    layers = [SubLayer(140, 4, 264, 520, False, seed=s, iters=2) for s in (1, 2, 3)]
    want = []
    for L in layers:
        L.forward()
        want.append({k: v.clone() for k, v in L.backward(L.kept["x"], L.kept["y"], L.kept["h_in"]).items()})
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(device()) for _ in layers]
    got = [None] * len(layers)
    for _ in range(3):
        for i, (L, s) in enumerate(zip(layers, streams)):
            with torch.cuda.stream(s):
                got[i] = L.backward(L.kept["x"], L.kept["y"], L.kept["h_in"])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(g[k].view(torch.uint8), w[k].view(torch.uint8)) for k in w)


def test_pointers_that_are_not_aligned_are_refused():
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    print("[case] alignment", file=sys.stderr, flush=True)
    buf = torch.zeros(4 * 64 + 8, dtype=torch.bfloat16, device=dev)
    x = buf[1:1 + 4 * 64].view(4, 64)
    w = torch.zeros((64, 64), dtype=torch.bfloat16, device=dev)
    for call in (lambda: mhc.mhc_checkpoint(x), lambda: mhc.mhc_glu(x, w, w), lambda: mhc.mhc_glu_backward(x, buf[:256].view(4, 64), w, w)):
        with pytest.raises(mhc.MhcError) as err:
            call()
        assert err.value.status == mhc.MHC_ERR_PARAM_INVALID


def test_tensors_of_more_than_2_to_the_32_values():
    # the last rows of a tensor whose offsets pass 32 bits give what they give by themselves
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    g = torch.Generator(device=dev).manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev).to(torch.bfloat16)
    for D in (7168, 7144):                                                   # whole blocks, and a shorter last one
        print(f"[case] checkpoint of 2^32 values D={D}", file=sys.stderr, flush=True)
        rows = (1 << 32) // D + 70
        x = torch.zeros((rows, D), dtype=torch.bfloat16, device=dev)
        x[-64:] = rnd(64, D)
        ck, small = mhc.mhc_checkpoint(x), mhc.mhc_checkpoint(x[-64:].contiguous())
        assert torch.equal(ck.codes[-64:], small.codes) and torch.equal(ck.scales[-64:], small.scales)
        assert not ck.codes[:4].any()
        assert torch.equal(mhc.mhc_checkpoint_restore(ck)[-64:], mhc.mhc_checkpoint_restore(small))
        del x, ck
    print("[case] post of 2^32 values", file=sys.stderr, flush=True)
    n, D = 8, 7168
    T = (1 << 32) // (n * D) + 9
    go, r = torch.zeros((T, n, D), dtype=torch.bfloat16, device=dev), torch.zeros((T, n, D), dtype=torch.bfloat16, device=dev)
    x, post, comb = torch.zeros((T, D), dtype=torch.bfloat16, device=dev), torch.rand((T, n), device=dev), torch.rand((T, n, n), device=dev)
    go[-5:], r[-5:], x[-5:] = rnd(5, n, D), rnd(5, n, D), rnd(5, D)
    tail = [t[-5:].contiguous() for t in (go, x, r, post, comb)]
    for kept in (False, True):
        whole = mhc.mhc_post_backward(go, x, mhc.mhc_checkpoint(r) if kept else r, post, comb)
        small = mhc.mhc_post_backward(tail[0], tail[1], mhc.mhc_checkpoint(tail[2]) if kept else tail[2], tail[3], tail[4])
        for k in whole:
            assert torch.equal(whole[k][-5:], small[k]), k
        del whole
    out, ck = mhc.mhc_post_checkpoint(x, r, post, comb)
    o2, c2 = mhc.mhc_post_checkpoint(tail[1], tail[2], tail[3], tail[4])
    assert torch.equal(out[-5:], o2) and torch.equal(ck.codes[-5:], c2.codes) and torch.equal(ck.scales[-5:], c2.scales)
    del go, r, out, ck
    print("[case] glu of 2^32 values", file=sys.stderr, flush=True)
    T, D, F = 40000, 8, 65536
    x, wg, wu = rnd(T, D), rnd(F, D), rnd(F, D)
    gh = torch.zeros((T, F), dtype=torch.bfloat16, device=dev)
    gh[-100:] = rnd(100, F)
    got = mhc.mhc_glu_backward(gh, x, wg, wu, need_h=True)
    small = mhc.mhc_glu_backward(gh[-100:].contiguous(), x[-100:].contiguous(), wg, wu, need_h=True)
    assert torch.equal(got["h"][-100:], mhc.mhc_glu(x, wg, wu)[-100:]) and torch.equal(got["h"][-100:], small["h"])
    # sums over f, and over tokens of which all but the last are zero, in other groupings: fp32 sums of at most 65536 and 100 terms,
    # then one rounding each (a step, 2^-7, apart at most where they fall on either side of a tie, with 2^-12 of the
    # largest for what cancels)
    for k in ("grad_x", "grad_w_gate", "grad_w_up"):
        a, b = (got[k][-100:] if k == "grad_x" else got[k]).double(), small[k].double()
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -12 * b.abs().max()).all(), k
    assert not got["grad_x"][:-100].any()
