"""The routing's backward, softmax without renormalisation, for a router that is sure of its experts: the gradient at a chosen expert
is w_e g_e - s_e sum_j w_j g_j, a small difference of nearly equal terms, to fp32 rounding of that difference's own parts.

With the weights that are given, R the other (not chosen) experts' part of the softmax, S = sum_j w_j g_j and far the distance of the
lowest logit from the top: the chosen experts' terms are fp64, R is fp32's (each exponential's argument, of at most far, the
exponential and the sum of up to 1024 terms: (2 far + 40) 2^-24 of R), and s_e depends on it as s_e R does. So the error before the last
rounding is at most |s_e S| R (2 far + 40) 2^-24, with fp32's least steps as experts_helpers.route_backward has them, and fp64's own: S is
k rounded products and their sum, s_e two exponentials, a sum of at most 32 terms and a quotient, and two products and the difference
follow: (2 k + 40) 2^-53 of the terms' magnitudes. The result is rounded once."""
import sys

import numpy as np
import pytest

from experts_helpers import U
from gpu_helpers import device

pytestmark = pytest.mark.gpu


def expected(L, g, w, e):
    """The gradient and its error's bound but for the last rounding, in longer arithmetic than fp64: the scores' differences cancel."""
    L, g, w = (a.astype(np.longdouble) for a in (L, g, w))
    T, E = L.shape
    rows = np.arange(T)[:, None]
    x = np.exp(L - L.max(1, keepdims=True))
    s = x / x.sum(1, keepdims=True)
    chosen = np.zeros((T, E), bool)
    chosen[np.broadcast_to(rows, e.shape), e] = True
    R = np.where(chosen, 0, s).sum(1, keepdims=True)
    S = (w * g).sum(1, keepdims=True)
    want = -s * S
    np.add.at(want, (rows, e), w * g)
    far = np.where(np.isfinite(L), L.max(1, keepdims=True) - L, 0).max(1, keepdims=True)
    part = np.where(chosen, R, 1) * np.abs(s * S)
    lim = part * U * (2 * far + 40) + 2.0 ** -149 * (np.abs(S) + 0.5) + (2 * e.shape[1] + 40) * 2.0 ** -53 * np.abs(w * g).sum(1, keepdims=True)
    return want, lim, chosen


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("T,E,k", [(29, 2, 1), (64, 60, 1), (61, 60, 2), (33, 200, 4), (50, 256, 1), (17, 300, 2), (9, 1000, 20), (40, 64, 17)])
def test_gradient_of_a_sure_router(T, E, k, dtype):
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    print(f"[case] sure router T={T} E={E} k={k} {dtype}", file=sys.stderr, flush=True)
    rng = np.random.default_rng(T + E + k)
    dt = getattr(torch, dtype)
    for scale in (1.0, 2.5):
        # the chosen from 4 to 22 above the others, near to each other or far apart
        L = rng.standard_normal((T, E))
        for t in range(T):
            at = rng.permutation(E)[:k]
            L[t, at] = rng.uniform(4, 22) + (rng.standard_normal(k) if t % 2 else rng.uniform(0, 1e-3, k))
        L[rng.random((T, E)) < 0.05] = -np.inf
        logits = torch.from_numpy(L.astype(np.float32)).to(dt)
        L = logits.double().numpy()
        g = rng.standard_normal((T, k)).astype(np.float32)
        g[::3] = g[::3, :1]                                  # equal gradients: what is left is the others' part alone
        w, e = mhc.mhc_route(logits.to(dev), k, renormalise=False, scale=scale)
        we, ee = w.cpu().numpy(), e.cpu().numpy()
        assert (ee >= 0).all()
        got = mhc.mhc_route_backward(torch.from_numpy(g).to(dev), logits.to(dev), w, e, renormalise=False, scale=scale).double().cpu().numpy()
        want, lim, chosen = expected(L, g, we, ee)
        # one rounding to the logits' format
        eps, least = {"float32": (U, 2.0 ** -150), "bfloat16": (2.0 ** -8, 2.0 ** -134), "float16": (2.0 ** -11, 2.0 ** -25)}[dtype]
        lim = lim + np.maximum(eps * (np.abs(want) + lim), least)
        err = np.abs(got - want)
        assert (err <= lim).all(), (dtype, scale, float((err / lim).max()), float((err / lim)[chosen].max()))
