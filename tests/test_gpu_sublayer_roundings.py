"""A sub-layer's training step against differentiation in 64 bits that rounds where the operators' documentation says they round
(h_in, h, y and the result of the forward; the gradients of y, of the residual path, of h, of the two projections and of h_in):
what is left between the two is each result's own rounding, and fp32 sums.

Tolerance, relative to a gradient's norm, with e = eps / 2 of the 16-bit format: a result's own rounding is at most e of every
value, so e of the norm. An intermediate's fp32 error moves its rounding to the other side only where the 64-bit value lies that close
to a tie. Sums of at most 520 terms of random sign are off by some sqrt(520) 2^-24 < 2^-19 of their size, 2^-9 of fp16's step
(2^-12 of bf16's), so that some 2^-8 of the values lie that close on either side; a step is 2 e, and 2^-8 of the values off by one are
2^-4 2 e of the norm. Ten such intermediates: sqrt(10) 2^-3 e < 0.4 e. 2 e bounds both together. A step that left out any one
of these roundings, or rounded anywhere else, would still pass; a wrong term of 1 % (bf16; 0.1 % in fp16) would not."""
import sys

import pytest

from test_gpu_sublayer import SubLayer

pytestmark = pytest.mark.gpu


def reference(L):
    import torch
    dt, n, T = L.x.dtype, L.n, L.x.shape[0]

    class Rounded(torch.autograd.Function):
        """The value, its gradient, or both rounded to the 16-bit format."""
        @staticmethod
        def forward(ctx, v, value, grad):
            ctx.grad = grad
            return v.to(dt).double() if value else v.clone()

        @staticmethod
        def backward(ctx, g):
            return g.to(dt).double() if ctx.grad else g, None, None

    both, grad_only = (lambda v: Rounded.apply(v, True, True)), (lambda v: Rounded.apply(v, False, True))
    d = lambda t: t.double().requires_grad_()
    x, phi, alpha, bias, gamma, wg, wu, wd = (d(t) for t in (L.x, L.phi, L.alpha, L.bias, L.gamma, L.wg, L.wu, L.wd))
    xf = x.reshape(T, -1)
    w = (xf * gamma.reshape(-1)) @ phi.t() * torch.rsqrt(xf.square().mean(1, keepdim=True) + 1e-6)
    h_pre = torch.sigmoid(alpha[0] * w[:, :n] + bias[:n]) + 1e-6
    h_post = 2 * torch.sigmoid(alpha[1] * w[:, n:2 * n] + bias[n:2 * n])
    a = torch.softmax((alpha[2] * w[:, 2 * n:] + bias[2 * n:]).reshape(T, n, n), -1) + 1e-6
    for k in range(1, 2 * L.iters):
        a = a / (a.sum(1 if k % 2 else 2, keepdim=True) + 1e-6)
    h_in = both((h_pre[:, :, None] * x).sum(1))
    g, u = grad_only(h_in @ wg.t()), grad_only(h_in @ wu.t())
    h = both(g * torch.sigmoid(g) * u)
    y = both(h @ wd.t())
    out = h_post[:, :, None] * y[:, None, :] + (a[:, :, :, None] * grad_only(x)[:, :, None, :]).sum(1)
    (out * L.grad_out.double()).sum().backward()
    return dict(grad_x=x.grad, grad_phi=phi.grad, grad_alpha=alpha.grad, grad_bias=bias.grad, grad_gamma=gamma.grad, grad_w_gate=wg.grad,
                grad_w_up=wu.grad, grad_w_down=wd.grad), out.detach()


@pytest.mark.parametrize("T,n,D,F,f16", [(200, 4, 264, 520, False), (97, 6, 136, 264, True), (130, 8, 96, 200, False), (40, 4, 264, 520, True)])
def test_training_step_with_its_roundings(T, n, D, F, f16):
    print(f"[case] sub-layer with roundings T={T} n={n} D={D} F={F} f16={f16}", file=sys.stderr, flush=True)
    L = SubLayer(T, n, D, F, f16, seed=T)
    out = L.forward()
    want, ref_out = reference(L)
    got = L.backward(L.x, L.y, L.h_in)
    e = 2.0 ** -11 if f16 else 2.0 ** -8
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())
    errs = {"out": rel(out, ref_out), **{k: rel(got[k], v) for k, v in want.items()}}
    assert all(v <= 2 * e for v in errs.values()), {k: v / e for k, v in errs.items()}
