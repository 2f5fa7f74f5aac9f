"""The training operators of an mHC sub-layer, case by case: what each computes, in plain form and by the library.

A sub-layer is  h_in = pre(streams),  y = F(h_in),  streams' = post(y, streams).  The operators:

  checkpoint       the streams [T, n, D] to 8 bits and back: one signed byte for each value and one power of two for
                   each run of 32 values along D
  post_checkpoint  hc_post that writes, beside the new streams, their 8-bit checkpoint
  post_backward    hc_post's gradients, from 16-bit activations or from their checkpoints
  pre_backward     the pre-mapping's gradients, from the streams' checkpoint
  glu              F's gated projection h = act(x Wg^T) (.) (x Wu^T)
  glu_backward     its gradients (and h again, for the gradient of the projection behind it), x in 16 bits or a checkpoint
"""
import math

import torch

own = False   # False: the plain forms below; True: the library's operators

_DT = {"bf16": torch.bfloat16, "f16": torch.float16}
_BLOCK = 32   # values that share one power of two


def listed():
    return [
        # the streams of the smallest workload, in fp16: the launches' own cost
        {"name": "checkpoint_tiny_f16", "op": "checkpoint", "T": 128, "n": 4, "D": 256, "dtype": "f16"},
        # one layer's streams of the large prefill, kept for the backward pass
        {"name": "checkpoint_large", "op": "checkpoint", "T": 16384, "n": 4, "D": 7168, "dtype": "bf16"},
        # the step from one layer to the next while training: an odd token count, a last block of 8 values, six streams
        {"name": "post_checkpoint_ragged_n6_f16", "op": "post_checkpoint", "T": 1003, "n": 6, "D": 1000, "dtype": "f16"},
        {"name": "post_checkpoint_mid", "op": "post_checkpoint", "T": 4096, "n": 4, "D": 4096, "dtype": "bf16"},
        # hc_post's backward without checkpoints, ragged, in fp16; and at the large prefill from checkpoints
        {"name": "post_backward_ragged_n6_f16", "op": "post_backward", "T": 1003, "n": 6, "D": 1000, "dtype": "f16",
         "ckpt": False},
        {"name": "post_backward_large_ckpt", "op": "post_backward", "T": 16384, "n": 4, "D": 7168, "dtype": "bf16",
         "ckpt": True},
        # the pre-mapping's backward from the streams' checkpoint: the mid prefill with gamma and the gradient that comes
        # past the sub-layer, and the large prefill
        {"name": "pre_backward_mid_ckpt_gamma", "op": "pre_backward", "T": 4096, "n": 4, "D": 4096, "dtype": "bf16",
         "gamma": True, "x_post": True, "iters": 20},
        {"name": "pre_backward_large_ckpt", "op": "pre_backward", "T": 16384, "n": 4, "D": 7168, "dtype": "bf16",
         "gamma": False, "x_post": False, "iters": 20},
        # serving: one token through the gated projection, bound by reading the weights
        {"name": "glu_one_token", "op": "glu", "T": 1, "D": 7168, "F": 14336, "dtype": "bf16", "act": "silu"},
        # a prefill's gated projection, bound by the matrix cores
        {"name": "glu_prefill", "op": "glu", "T": 16384, "D": 4096, "F": 16384, "dtype": "bf16", "act": "silu"},
        # a small model's training step with a ragged batch, tanh-GELU, fp16, x kept in 16 bits
        {"name": "glu_backward_ragged_f16", "op": "glu_backward", "T": 1003, "D": 2048, "F": 5464, "dtype": "f16",
         "act": "gelu_tanh", "ckpt": False},
        # a large model's training step from the checkpoint of x
        {"name": "glu_backward_large_ckpt", "op": "glu_backward", "T": 8192, "D": 7168, "F": 14336, "dtype": "bf16",
         "act": "silu", "ckpt": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["checkpoint", "post_checkpoint", "post_backward", "pre_backward", "glu", "glu_backward"])
    c = {"op": op, "T": _log(rng, 1, 16384), "D": 8 * _log(rng, 4, 1024), "dtype": rng.choice(["bf16", "bf16", "f16"])}
    if op in ("glu", "glu_backward"):
        c["F"] = 8 * _log(rng, 4, 2048)
        c["act"] = rng.choice(["silu", "gelu_tanh"])
        most = 16384 * 4096 * 16384 if op == "glu" else 8192 * 7168 * 14336
        c["T"] = max(1, min(c["T"], most // (c["D"] * c["F"])))
    else:
        c["n"] = rng.choice([4, 6, 8])
        c["T"] = max(1, min(c["T"], 16384 * 4 * 7168 // (c["n"] * c["D"])))
    if op in ("post_backward", "glu_backward"):
        c["ckpt"] = rng.random() < 0.6
    if op == "pre_backward":
        c["gamma"] = rng.random() < 0.5
        c["x_post"] = rng.random() < 0.5
        c["iters"] = rng.choice([0, 1, 5, 20, 20])
    return c


# ---------------------------------------------------------------------------------------------------- inputs


def _dev():
    return torch.device("cuda", 0)


class _Gen:
    def __init__(self, seed):
        self.g = torch.Generator(device=_dev()).manual_seed(int(seed))

    def randn(self, *shape, std=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=self.g, device=_dev(), dtype=torch.float32).mul_(std).to(dtype)

    def rand(self, *shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=self.g, device=_dev(), dtype=torch.float32) * (hi - lo) + lo


def _activation(g, *shape, dtype):
    # activations: normal, with channels of different sizes and a few large ones, as residual streams have
    D = shape[-1]
    size = torch.exp(g.randn(D, std=0.5))
    size = torch.where(g.rand(D) < 0.01, size * 8.0, size)
    return (g.randn(*shape) * size).to(dtype)


def _store(x):
    """The 8-bit checkpoint of x in elementary operations: codes (int8) and the blocks' exponents + 127 (uint8)."""
    low = -24 if x.dtype == torch.float16 else -126
    D = x.shape[-1]
    v = torch.nn.functional.pad(x.float(), (0, -D % _BLOCK)).unflatten(-1, (-1, _BLOCK))
    e = (torch.frexp(v.abs().amax(-1))[1].int() - 7).clamp_(min=low)
    q = torch.round(torch.ldexp(v, -e.unsqueeze(-1))).clamp_(-127, 127)
    return q.flatten(-2)[..., :D].to(torch.int8).contiguous(), (e + 127).to(torch.uint8)


def _load(codes, scales):
    """A checkpoint's values, in float32 (exact)."""
    step = torch.ldexp(torch.ones((), device=codes.device), scales.int() - 127)
    return codes.float() * step.repeat_interleave(_BLOCK, -1)[..., :codes.shape[-1]]


def _sinkhorn_planes(L, iters, eps):
    sums, mats = [], []
    for k in range(2 * iters):
        if k == 0:
            a = torch.exp(L - L.amax(-1, keepdim=True))
            s = a.sum(-1, keepdim=True)
            a = a / s + eps
        else:
            s = a.sum(-2 if k % 2 else -1, keepdim=True) + eps
            a = a / s
        sums.append(s.reshape(s.shape[0], -1))
        mats.append(a)
    return torch.stack(sums).float(), torch.stack(mats).float()


def prepare(case, seed):
    g, T, D, dt, op = _Gen(seed), case["T"], case["D"], _DT[case["dtype"]], case["op"]
    s = dict(case, dt=dt)
    if op in ("glu", "glu_backward"):
        F = case["F"]
        s["x"] = _activation(g, T, D, dtype=dt)
        # weights that keep the gate's input near unit size
        s["w_gate"] = g.randn(F, D, std=0.7 / math.sqrt(D), dtype=dt)
        s["w_up"] = g.randn(F, D, std=0.7 / math.sqrt(D), dtype=dt)
        if op == "glu_backward":
            s["grad_h"] = g.randn(T, F, dtype=dt)
            if case["ckpt"]:
                s["codes"], s["scales"] = _store(s.pop("x"))
        return s
    n = case["n"]
    streams = _activation(g, T, n, D, dtype=dt)
    if op == "checkpoint":
        s["x"] = streams
    elif op in ("post_checkpoint", "post_backward"):
        s["x"] = _activation(g, T, D, dtype=dt)
        s["residual"] = streams
        s["post"] = g.rand(T, n, lo=0.2, hi=1.8)
        s["comb"] = torch.softmax(g.randn(T, n, n), -1)
        if op == "post_backward":
            s["grad_out"] = g.randn(T, n, D, dtype=dt)
            if case["ckpt"]:
                s["codes"], s["scales"] = _store(s.pop("residual"))
                s["x_codes"], s["x_scales"] = _store(s.pop("x"))
    else:   # pre_backward: what the forward saved, and the gradients that come back
        M, K, eps = n * n + 2 * n, n * D, 1e-6
        phi = g.randn(M, K, std=1.0 / math.sqrt(K))
        gamma = g.rand(n, D, lo=0.5, hi=1.5) if case["gamma"] else None
        alpha = g.rand(3, lo=0.5, hi=1.5)
        bias = g.randn(M, std=0.1)
        xf = streams.reshape(T, K).float()
        inv = torch.rsqrt(xf.square().mean(-1) + 1e-6)
        mix = torch.mm(xf if gamma is None else xf * gamma.reshape(K), phi.t())
        w = mix * inv[:, None]
        s.update(phi=phi, gamma=gamma, alpha=alpha, eps=eps, inv_rms=inv, h_mix=mix,
                 h_pre=torch.sigmoid(alpha[0] * w[:, :n] + bias[:n]) + eps,
                 h_post=2 * torch.sigmoid(alpha[1] * w[:, n:2 * n] + bias[n:2 * n]))
        if case["iters"]:
            L = (alpha[2] * w[:, 2 * n:] + bias[2 * n:]).reshape(T, n, n).double()
            s["sum_out"], s["norm_out"] = _sinkhorn_planes(L, case["iters"], eps)
        s["codes"], s["scales"] = _store(streams)
        del xf, streams
        s["grad_h_in"] = g.randn(T, D, dtype=dt)
        s["grad_h_post"] = g.randn(T, n)
        s["grad_h_res"] = g.randn(T, n, n)
        s["grad_x_post"] = g.randn(T, n, D, dtype=dt) if case["x_post"] else None
    return s


# ---------------------------------------------------------------------------------------------------- one pass


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import mhc_hyper_connection_amd as mhc

    op = s["op"]
    if op == "checkpoint":
        return mhc.mhc_checkpoint_restore(mhc.mhc_checkpoint(s["x"]))
    if op == "post_checkpoint":
        out, ck = mhc.mhc_post_checkpoint(s["x"], s["residual"], s["post"], s["comb"])
        return {"out": out, "restored": mhc.mhc_checkpoint_restore(ck)}
    if op == "post_backward":
        x, residual = s.get("x"), s.get("residual")
        if s["ckpt"]:
            x = mhc.Checkpoint(s["x_codes"], s["x_scales"], s["dt"])
            residual = mhc.Checkpoint(s["codes"], s["scales"], s["dt"])
        return mhc.mhc_post_backward(s["grad_out"], x, residual, s["post"], s["comb"])
    if op == "pre_backward":
        return mhc.mhc_pre_backward(mhc.Checkpoint(s["codes"], s["scales"], s["dt"]), s["phi"], s["alpha"], s["grad_h_in"],
                                    s["grad_h_post"], s["grad_h_res"], s["inv_rms"], s["h_mix"], s["h_pre"], s["h_post"],
                                    s["gamma"], s["grad_x_post"], hc_eps=s["eps"], num_iters=s["iters"],
                                    sum_out=s.get("sum_out"), norm_out=s.get("norm_out"))
    if op == "glu":
        return mhc.mhc_glu(s["x"], s["w_gate"], s["w_up"], act=s["act"])
    x = mhc.Checkpoint(s["codes"], s["scales"], s["dt"]) if s["ckpt"] else s["x"]
    return mhc.mhc_glu_backward(s["grad_h"], x, s["w_gate"], s["w_up"], act=s["act"], need_h=True)


def _gate(g, act):
    """act(g) and act'(g): act(g) = g sigmoid(z), z = g or 2 sqrt(2 / pi) (g + 0.044715 g^3)."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    c = 2 * math.sqrt(2 / math.pi)
    s = torch.sigmoid(c * (g + 0.044715 * g * g * g))
    return g * s, s + g * s * (1 - s) * c * (1 + 3 * 0.044715 * g * g)


def _mix(comb, streams):
    # sum over comb's first index, in float32: comb[t, i, j] streams[t, i, d]
    return torch.bmm(comb.transpose(1, 2).contiguous(), streams)


def _run_plain(s):
    op, dt = s["op"], s["dt"]
    if op == "checkpoint":
        return _load(*_store(s["x"])).to(dt)
    if op == "post_checkpoint":
        out = (s["post"][:, :, None] * s["x"].float()[:, None, :] + _mix(s["comb"], s["residual"].float())).to(dt)
        return {"out": out, "restored": _load(*_store(out)).to(dt)}
    if op == "post_backward":
        x = _load(s["x_codes"], s["x_scales"]) if s["ckpt"] else s["x"].float()
        residual = _load(s["codes"], s["scales"]) if s["ckpt"] else s["residual"].float()
        go = s["grad_out"].float()
        return {"grad_x": torch.bmm(s["post"][:, None, :].contiguous(), go)[:, 0].to(dt),
                "grad_residual": torch.bmm(s["comb"], go).to(dt),
                "grad_post": (go * x[:, None, :]).sum(-1),
                "grad_comb": torch.bmm(residual, go.transpose(1, 2).contiguous())}
    if op == "pre_backward":
        return _pre_backward_plain(s)
    if op == "glu":
        x = s["x"].float()
        return (_gate(torch.mm(x, s["w_gate"].float().t()), s["act"])[0] * torch.mm(x, s["w_up"].float().t())).to(dt)
    x = _load(s["codes"], s["scales"]) if s["ckpt"] else s["x"].float()
    wg, wu, gh = s["w_gate"].float(), s["w_up"].float(), s["grad_h"].float()
    u = torch.mm(x, wu.t())
    a, da = _gate(torch.mm(x, wg.t()), s["act"])
    dg, du = gh * u * da, gh * a
    return {"grad_x": (torch.mm(dg, wg) + torch.mm(du, wu)).to(dt), "grad_w_gate": torch.mm(dg.t(), x).to(dt),
            "grad_w_up": torch.mm(du.t(), x).to(dt), "h": (a * u).to(dt)}


def _pre_backward_plain(s):
    dt, T, n, D = s["dt"], s["T"], s["n"], s["D"]
    K = n * D
    x = _load(s["codes"], s["scales"])                                   # [T, n, D]
    gh = s["grad_h_in"].float()
    G = s["grad_h_res"].double()
    if s["iters"]:   # back through the saved Sinkhorn planes: a recursion of 2 iters - 1 steps
        A, S = s["norm_out"].double(), s["sum_out"].double()
        for k in range(2 * s["iters"] - 1, 0, -1):
            ax = 1 if k % 2 else 2
            G = (G - (G * A[k]).sum(ax, keepdim=True)) / S[k].unsqueeze(ax)
        P = A[0] - s["eps"]
        G = P * (G - (G * P).sum(2, keepdim=True))
    ghp = (gh[:, None, :] * x).sum(-1).double()
    hp, hq, inv, mix = s["h_pre"].double() - s["eps"], s["h_post"].double(), s["inv_rms"].double(), s["h_mix"].double()
    terms = torch.cat([ghp * hp * (1 - hp), s["grad_h_post"].double() * hq * (1 - hq / 2), G.reshape(T, n * n)], 1)
    branch = s["alpha"].double().repeat_interleave(torch.tensor([n, n, n * n], device=x.device))
    gw = terms * branch
    tw = terms * mix * inv[:, None]
    gmix = (gw * inv[:, None]).float()
    c3 = ((gw * mix).sum(1) * inv ** 3 / K).float()
    xrs = torch.mm(gmix, s["phi"]).reshape(T, n, D)
    gphi = torch.mm(gmix.t().contiguous(), x.reshape(T, K))
    gx = gh[:, None, :] * s["h_pre"][:, :, None] - c3[:, None, None] * x
    out = {"grad_alpha": torch.stack([tw[:, :n].sum(), tw[:, n:2 * n].sum(), tw[:, 2 * n:].sum()]).float(),
           "grad_bias": terms.sum(0).float()}
    if s["gamma"] is not None:
        gx = gx + xrs * s["gamma"]
        out["grad_gamma"] = (x * xrs).sum(0)
        gphi = gphi * s["gamma"].reshape(K)
    else:
        gx = gx + xrs
    if s["grad_x_post"] is not None:
        gx = gx + s["grad_x_post"].float()
    return dict(out, grad_x=gx.to(dt), grad_phi=gphi)


# ---------------------------------------------------------------------------------------------------- work


def work(case):
    T, D, op = case["T"], case["D"], case["op"]
    if op in ("glu", "glu_backward"):
        F = case["F"]
        w = 2 * 2 * F * D
        if op == "glu":
            return {"bytes": 2 * T * D + w + 2 * T * F, "flops": 4 * T * D * F}
        x = T * (D + -(-D // _BLOCK)) if case["ckpt"] else 2 * T * D
        return {"bytes": x + 2 * w + 2 * T * F + 2 * T * D + 2 * T * F, "flops": 12 * T * D * F}
    n = case["n"]
    el = T * n * D
    ck = T * n * (D + -(-D // _BLOCK))
    gates = 4 * T * (n + n * n)
    if op == "checkpoint":          # x in, the checkpoint out; the checkpoint in, x out
        return {"bytes": 2 * el + ck + ck + 2 * el, "flops": 4 * el}
    if op == "post_checkpoint":     # ... and the checkpoint restored
        return {"bytes": 2 * T * D + 2 * el + gates + 2 * el + ck + ck + 2 * el, "flops": 2 * el * (n + 1)}
    if op == "post_backward":
        acts = ck + T * (D + -(-D // _BLOCK)) if case["ckpt"] else 2 * el + 2 * T * D
        return {"bytes": 2 * el + acts + gates + 2 * el + 2 * T * D + gates, "flops": 4 * el * (n + 1)}
    M, K, it = n * n + 2 * n, n * D, case["iters"]
    b = ck + 2 * T * D + 2 * el + 4 * T * (n + n * n + 1 + M + 2 * n) + 8 * M * K + 24 + 4 * M
    b += (8 * K if case["gamma"] else 0) + (2 * el if case["x_post"] else 0) + 8 * it * T * (n + n * n)
    return {"bytes": b, "flops": 4 * T * M * K + 6 * el}


# ---------------------------------------------------------------------------------------------------- 64 bits


def _exact_store(v):
    """The values that the checkpoint of the 16-bit tensor v stands for, from the definition: per run of 32 values the
    step 2^e with e = floor(log2 max|v|) - 6 (not below the format's least), each value the nearest multiple, ties to the
    even one, at most 127 steps."""
    least = 2.0 ** (-24 if v.dtype == torch.float16 else -126)
    d = v.double()
    out = torch.empty_like(d)
    D = v.shape[-1]
    whole = D // _BLOCK * _BLOCK
    for lo, hi in ((0, whole), (whole, D)):
        if hi > lo:
            b = d[..., lo:hi].reshape(*d.shape[:-1], -1, min(_BLOCK, hi - lo))
            top = b.abs().max(-1, keepdim=True).values
            step = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -140))) - 6).clamp(min=least)
            r = b / step
            f = torch.floor(r)
            odd = torch.remainder(f, 2)
            r = f + ((r - f > 0.5) | ((r - f == 0.5) & (odd == 1))).double()
            out[..., lo:hi] = (r.clamp(-127, 127) * step).reshape(*d.shape[:-1], hi - lo)
    return out


def _kept(s, codes, scales, name):
    if not s.get("ckpt", True):
        return s[name].double()
    c, e = s[codes].double(), s[scales].double()
    at = torch.arange(c.shape[-1], device=c.device) // _BLOCK
    return c * torch.exp2(e - 127.0)[..., at]


def exact(case, seed):
    s = prepare(case, seed)
    op, dt = s["op"], s["dt"]
    if op == "checkpoint":
        return _exact_store(s["x"])
    if op in ("post_checkpoint", "post_backward"):
        post, comb = s["post"].double(), s["comb"].double()
        if op == "post_checkpoint":
            x, r = s["x"].double(), s["residual"].double()
            out = torch.stack([post[:, j, None] * x + sum(comb[:, i, j, None] * r[:, i] for i in range(s["n"]))
                               for j in range(s["n"])], 1)
            return {"out": out, "restored": _exact_store(out.to(dt))}
        x, r = _kept(s, "x_codes", "x_scales", "x"), _kept(s, "codes", "scales", "residual")
        go, n = s["grad_out"].double(), s["n"]
        return {"grad_x": sum(post[:, j, None] * go[:, j] for j in range(n)),
                "grad_residual": torch.stack([sum(comb[:, i, j, None] * go[:, j] for j in range(n)) for i in range(n)], 1),
                "grad_post": torch.stack([(go[:, j] * x).sum(-1) for j in range(n)], 1),
                "grad_comb": torch.stack([torch.stack([(r[:, i] * go[:, j]).sum(-1) for j in range(n)], 1)
                                          for i in range(n)], 1)}
    if op == "pre_backward":
        return _pre_backward_exact(s)
    x = _kept(s, "codes", "scales", "x") if op == "glu_backward" else s["x"].double()
    wg, wu = s["w_gate"].double(), s["w_up"].double()
    g, u = x @ wg.t(), x @ wu.t()
    if s["act"] == "silu":
        q = 1 / (1 + torch.exp(-g))
        a, da = g * q, q * (1 + g * (1 - q))
    else:
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g ** 3))
        a, da = 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    if op == "glu":
        return a * u
    gh = s["grad_h"].double()
    out = {"h": a * u}
    da *= gh
    da *= u
    del g, u
    a *= gh
    return dict(out, grad_x=da @ wg + a @ wu, grad_w_gate=da.t() @ x, grad_w_up=a.t() @ x)


def _pre_backward_exact(s):
    T, n, D, eps, al = s["T"], s["n"], s["D"], s["eps"], s["alpha"].double()
    x = _kept(s, "codes", "scales", "x").reshape(T, n * D)
    gh, hp = s["grad_h_in"].double(), s["h_pre"].double()
    q, inv, mix = s["h_post"].double(), s["inv_rms"].double().unsqueeze(1), s["h_mix"].double()
    g_pre = torch.stack([(x[:, i * D:(i + 1) * D] * gh).sum(1) for i in range(n)], 1) * (hp - eps) * (1 - hp + eps)
    g_post = s["grad_h_post"].double() * (q - q * q / 2)
    G = s["grad_h_res"].double()
    for k in range(2 * s["iters"] - 1, -1, -1):
        A, S = s["norm_out"][k].double(), s["sum_out"][k].double()
        if k == 0:      # a softmax along the rows
            A = A - eps
            G = A * G - A * (A * G).sum(-1, keepdim=True)
        elif k % 2:     # a division of the columns by their sums
            G = (G - torch.ones_like(A[:, :, :1]) * (G * A).sum(1, keepdim=True)) / S[:, None, :]
        else:
            G = (G - (G * A).sum(2, keepdim=True)) / S[:, :, None]
    g_res = G.reshape(T, n * n)
    w = mix * inv
    out = {"grad_bias": torch.cat([g_pre.sum(0), g_post.sum(0), g_res.sum(0)]),
           "grad_alpha": torch.stack([(g_pre * w[:, :n]).sum(), (g_post * w[:, n:2 * n]).sum(), (g_res * w[:, 2 * n:]).sum()])}
    gw = torch.cat([al[0] * g_pre, al[1] * g_post, al[2] * g_res], 1)
    back = (gw * inv) @ s["phi"].double()
    gphi = (gw * inv).t() @ x
    if s["gamma"] is not None:
        ga = s["gamma"].double().reshape(1, -1)
        out["grad_gamma"] = (back * x).sum(0).reshape(n, D)
        back *= ga
        gphi *= ga
    back -= (gw * mix).sum(1, keepdim=True) * inv ** 3 / (n * D) * x
    gx = back.reshape(T, n, D)
    gx += gh.unsqueeze(1) * hp.unsqueeze(2)
    if s["grad_x_post"] is not None:
        gx += s["grad_x_post"].double()
    return dict(out, grad_x=gx, grad_phi=gphi)
