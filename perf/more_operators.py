"""The operators of an mHC sub-layer whose F is a mixture of experts, case by case: what each computes, in plain form and by
the library.

  route           the experts of each token and their weights from the router's logits, and the plan: the pairs
                  (token, slot) sorted by expert, which the experts' products read
  route_backward  the logits' gradient from the weights'
  mxfp4           16-bit rows to microscaled 4-bit floats (e2m1 codes, one power of two for each 32 values) and back
  product         y = x w^T with 4-bit weights; x in 16 bits, which the call quantises
  experts_glu     the experts' gated projection over 4-bit weights
  experts_down    the experts' projection back over 4-bit weights, and the sum of each token's results by its weights
"""
import math

import torch

own = False   # False: the plain forms below; True: the library's operators

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BLOCK = 32   # values that share one power of two
_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # of e2m1's codes 0 .. 7; codes 8 .. 15 are their negatives


def listed():
    return [
        # serving: one token's routing, the launches' own cost
        {"name": "route_one_token", "op": "route", "T": 1, "E": 128, "k": 8, "dtype": "f32", "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "renorm": True, "scale": 1.0, "masked": False},
        # a large prefill: sigmoid scores, a bias that balances the experts, 4 of 8 groups
        {"name": "route_large_groups", "op": "route", "T": 16384, "E": 256, "k": 8, "dtype": "f32", "score": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "renorm": True, "scale": 2.5, "masked": False},
        # training: a ragged batch of a small model, bf16 logits, an odd number of experts, padded tokens, weights not
        # renormalised (then every logit has a gradient); and a large model's
        {"name": "route_backward_ragged_bf16", "op": "route_backward", "T": 1003, "E": 60, "k": 4, "dtype": "bf16",
         "score": "softmax", "bias": False, "groups": 1, "top_groups": 1, "renorm": False, "scale": 1.0, "masked": True},
        {"name": "route_backward_large", "op": "route_backward", "T": 16384, "E": 256, "k": 8, "dtype": "f32",
         "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "renorm": True, "scale": 2.5, "masked": False},
        # activations of a ragged batch whose last block is short, in fp16; and a large prefill's
        {"name": "mxfp4_ragged_f16", "op": "mxfp4", "T": 1003, "D": 1000, "dtype": "f16"},
        {"name": "mxfp4_large", "op": "mxfp4", "T": 16384, "D": 7168, "dtype": "bf16"},
        # serving: one token, bound by reading the weights; and a prefill, bound by the matrix cores
        {"name": "product_one_token", "op": "product", "T": 1, "K": 7168, "N": 16384, "dtype": "bf16"},
        {"name": "product_prefill", "op": "product", "T": 16384, "K": 4096, "N": 16384, "dtype": "bf16"},
        # serving: one token through its 8 of 64 experts; and a prefill's tokens through all of them
        {"name": "experts_glu_one_token", "op": "experts_glu", "T": 1, "E": 64, "k": 8, "D": 7168, "F": 2048,
         "dtype": "bf16", "act": "silu", "masked": False},
        {"name": "experts_glu_prefill", "op": "experts_glu", "T": 8192, "E": 64, "k": 8, "D": 4096, "F": 2048,
         "dtype": "bf16", "act": "silu", "masked": False},
        # a ragged batch of a small model in fp16, padded tokens, a reduction that ends inside a block; and the prefill
        {"name": "experts_down_ragged_f16", "op": "experts_down", "T": 1003, "E": 20, "k": 4, "D": 2048, "F": 5464,
         "dtype": "f16", "masked": True},
        {"name": "experts_down_prefill", "op": "experts_down", "T": 8192, "E": 64, "k": 8, "D": 4096, "F": 2048,
         "dtype": "bf16", "masked": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "mxfp4", "product", "experts_glu", "experts_down"])
    c = {"op": op, "T": _log(rng, 1, 16384), "dtype": rng.choice(["bf16", "bf16", "f16"])}
    if op == "mxfp4":
        c["D"] = _log(rng, 8, 8192)
        c["T"] = max(1, min(c["T"], 16384 * 7168 // c["D"]))
        return c
    if op == "product":
        c["K"], c["N"] = 8 * _log(rng, 4, 1024), 8 * _log(rng, 4, 2048)
        c["T"] = max(1, min(c["T"], 16384 * 4096 * 16384 // (c["K"] * c["N"])))
        return c
    c["masked"] = rng.random() < 0.3
    if op in ("route", "route_backward"):
        c["dtype"] = rng.choice(["f32", "f32", "bf16", "f16"])
        c["groups"] = rng.choice([1, 1, 2, 4, 8])
        per = _log(rng, 2, 512 // c["groups"])
        c["E"] = c["groups"] * per
        c["top_groups"] = rng.randint(1, c["groups"])
        c["k"] = rng.randint(1, min(16, c["top_groups"] * per))
        c["score"] = rng.choice(["softmax", "sigmoid"])
        c["bias"] = rng.random() < 0.6
        c["renorm"] = rng.random() < 0.6
        c["scale"] = rng.choice([1.0, 2.5])
        c["T"] = max(1, min(c["T"], 16384 * 256 // c["E"]))
        return c
    c["E"] = _log(rng, 2, 64)
    c["k"] = rng.randint(1, min(8, c["E"]))
    c["D"], c["F"] = 8 * _log(rng, 4, 900), 8 * _log(rng, 4, 700)
    c["E"] = max(c["k"], min(c["E"], 64 * 7168 * 2048 // (c["D"] * c["F"])))
    c["T"] = max(1, min(c["T"], 8192 * 8 * 4096 * 2048 // (c["k"] * c["D"] * c["F"]), 8192 * 8 * 4096 // (c["k"] * max(c["D"], c["F"]))))
    if op == "experts_glu":
        c["act"] = rng.choice(["silu", "gelu_tanh"])
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
    """x [..., D] as microscaled 4-bit floats, in elementary operations: codes uint8 [..., 16 ceil(D / 32)], two to a byte,
    the even value's in the low half; scales uint8 [..., 4 ceil(D / 128)], a block's power of two + 127; zeros behind D.
    With a the block's largest magnitude, rounded to one bit behind its leading one, the power is floor(log2 a) - 2: a then
    falls on 4 or 6 steps. It stops where 6 steps are still finite in x's format."""
    top = 140 if x.dtype == torch.float16 else 252
    D = x.shape[-1]
    v = torch.nn.functional.pad(x.float(), (0, -D % _BLOCK)).unflatten(-1, (-1, _BLOCK))
    a = v.abs().amax(-1)
    s = (((a.view(torch.int32) + (1 << 21)) >> 23) - 2).clamp_(0, top)
    r = torch.ldexp(v.abs(), (127 - s).unsqueeze(-1))
    step = torch.where(r < 2, 0.5, torch.where(r < 4, 1.0, 2.0))
    r = (torch.round(r / step) * step).clamp_(max=6.0)
    c = torch.where(r < 2, 2 * r, torch.where(r < 4, r + 2, r / 2 + 4)).to(torch.uint8)
    c += (v < 0).to(torch.uint8) * 8
    bad = ~torch.isfinite(a)
    c[bad] = 0
    s = torch.where(bad, 255, s)
    c = c.flatten(-2)
    codes = (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous()
    return codes, torch.nn.functional.pad(s.to(torch.uint8), (0, -s.shape[-1] % 4)).contiguous()


def _load(codes, scales, D):
    """The values that codes and scales stand for, in float32 (exact)."""
    table = torch.tensor(_VALUES + tuple(-v for v in _VALUES), device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)[..., :D]
    step = torch.ldexp(torch.ones((), device=codes.device), scales.int() - 127)
    step = torch.where(scales == 255, torch.nan, step)
    return table[c.int()] * step.repeat_interleave(_BLOCK, -1)[..., :D]


def _weights(g, *shape):
    # 4-bit weights, a matrix at a time; of a size that keeps results near unit size
    one = lambda: _store(g.randn(*shape[-2:], std=0.7 / math.sqrt(shape[-1]), dtype=torch.bfloat16))  # noqa: E731
    if len(shape) == 2:
        return one()
    both = [one() for _ in range(shape[0])]
    return torch.stack([c for c, _ in both]), torch.stack([s for _, s in both])


def _some_experts(g, T, E, k, masked):
    # each token's experts and weights, some experts more popular than others; padded tokens have none
    logits = g.randn(T, E) + g.randn(E, std=0.5)
    v, e = torch.topk(logits, k, -1)
    w, e = torch.softmax(v, -1), e.int()
    if masked:
        pad = g.rand(T) < 0.2
        w[pad], e[pad] = 0.0, -1
    return w, e


def _plan(experts, E):
    """Where each expert's pairs begin, and the pairs (their places in `experts`) sorted by expert, those without one last."""
    e = experts.reshape(-1).long()
    e = torch.where(e < 0, E, e)
    pairs = torch.sort(e, dim=-1, stable=True)[1]
    begin = torch.searchsorted(e[pairs], torch.arange(E + 1, device=e.device))
    return begin.int(), pairs.int()


def prepare(case, seed):
    g, T, dt, op = _Gen(seed), case["T"], _DT[case["dtype"]], case["op"]
    s = dict(case, dt=dt)
    if op == "mxfp4":
        s["x"] = _activation(g, T, case["D"], dtype=dt)
    elif op == "product":
        s["x"] = _activation(g, T, case["K"], dtype=dt)
        s["w"] = _weights(g, case["N"], case["K"])
    elif op in ("route", "route_backward"):
        E = case["E"]
        logits = g.randn(T, E, std=1.5)
        if case["masked"]:   # experts that a token may not have, and padded tokens
            logits = torch.where(g.rand(T, E) < 0.1, -math.inf, logits)
            logits[g.rand(T) < 0.1] = -math.inf
        s["logits"] = logits.to(dt)
        # a balance bias in steps of a training run's updates, so that two experts may have the same
        s["route_bias"] = torch.round(g.randn(E, std=0.05) * 1000) / 1000 if case["bias"] else None
        if op == "route_backward":
            s["weights"], s["experts"] = _route(s)
            s["grad_weights"] = g.randn(T, case["k"])
    else:
        E, k, D, F = case["E"], case["k"], case["D"], case["F"]
        s["weights"], s["experts"] = _some_experts(g, T, E, k, case["masked"])
        s["offsets"], s["pairs"] = _plan(s["experts"], E)
        if op == "experts_glu":
            s["x"] = _activation(g, T, D, dtype=dt)
            s["w_gate"], s["w_up"] = _weights(g, E, F, D), _weights(g, E, F, D)
        else:
            u = g.randn(T, k, F, std=0.7)
            s["h"] = (u * torch.sigmoid(u) * g.randn(T, k, F, std=0.7)).to(dt)
            s["w_down"] = _weights(g, E, D, F)
    return s


# ---------------------------------------------------------------------------------------------------- one pass


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import mhc_hyper_connection_amd as mhc

    op = s["op"]
    if op == "route":
        weights, experts = mhc.mhc_route(s["logits"], s["k"], bias=s["route_bias"], score=s["score"], groups=s["groups"],
                                         top_groups=s["top_groups"], renormalise=s["renorm"], scale=s["scale"])
        plan = mhc.mhc_experts_plan(experts, s["E"])
        return {"weights": weights, "experts": experts, "offsets": plan.offsets, "pairs": plan.pairs}
    if op == "route_backward":
        return mhc.mhc_route_backward(s["grad_weights"], s["logits"], s["weights"], s["experts"], score=s["score"],
                                      renormalise=s["renorm"], scale=s["scale"])
    if op == "mxfp4":
        return mhc.mhc_mxfp4_restore(mhc.mhc_mxfp4(s["x"]))
    if op == "product":
        return mhc.mhc_mxfp4_product(s["x"], mhc.Mxfp4(*s["w"], s["dt"], s["K"]))
    plan = mhc.ExpertsPlan(s["offsets"], s["pairs"], (s["T"], s["k"]))
    if op == "experts_glu":
        return mhc.mhc_experts_glu(s["x"], plan, mhc.Mxfp4(*s["w_gate"], s["dt"], s["D"]),
                                   mhc.Mxfp4(*s["w_up"], s["dt"], s["D"]), act=s["act"])
    return mhc.mhc_experts_down(s["h"], plan, s["weights"], mhc.Mxfp4(*s["w_down"], s["dt"], s["F"]))


def _scores(s):
    L = s["logits"].double()
    if s["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-L))
    top = L.amax(-1, keepdim=True)
    p = torch.exp(L - torch.where(torch.isfinite(top), top, 0.0))
    return p / p.sum(-1, keepdim=True).clamp(min=1e-300)   # a row that is masked throughout: zeros


def _route(s):
    """Weights and experts. Scores in 64 bits: two experts may be nearer to each other than 32 tell."""
    T, E, k, G = s["T"], s["E"], s["k"], s["groups"]
    score = _scores(s)
    # the order of the choice: score + bias, or the logits, which order the scores
    choice = s["logits"].double() if s["route_bias"] is None else score + s["route_bias"].double()
    off = torch.isneginf(s["logits"])
    choice = choice.masked_fill(off, -math.inf)
    if G > 1:
        value = (score if s["route_bias"] is None else choice).masked_fill(off, -math.inf).reshape(T, G, E // G)
        best = torch.sort(value, dim=-1, descending=True)[0][..., :2]
        group = torch.where(best > -math.inf, best, 0.0).sum(-1).masked_fill(best[..., 0] == -math.inf, -math.inf)
        keep = torch.sort(group, dim=-1, descending=True, stable=True)[1][:, :s["top_groups"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=keep.device).scatter_(1, keep, True)
        choice = choice.masked_fill(~kept.repeat_interleave(E // G, 1), -math.inf)
    order = torch.sort(choice, dim=-1, descending=True, stable=True)
    experts = order[1][:, :k]
    w = score.gather(1, experts)
    none = order[0][:, :k] == -math.inf
    w = w.masked_fill(none, 0.0)
    if s["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return (w * s["scale"]).float(), experts.masked_fill(none, -1).int()


def _gate(g, act):
    """act(g) = g sigmoid(z), z = g or 2 sqrt(2 / pi) (g + 0.044715 g^3)."""
    return g * torch.sigmoid(g if act == "silu" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g))


def _run_plain(s):
    op, dt = s["op"], s["dt"]
    if op == "route":
        weights, experts = _route(s)
        offsets, pairs = _plan(experts, s["E"])
        return {"weights": weights, "experts": experts, "offsets": offsets, "pairs": pairs}
    if op == "route_backward":
        return _route_backward(s).to(dt)
    if op == "mxfp4":
        return _load(*_store(s["x"]), s["D"]).to(dt)
    if op == "product":
        K = s["K"]
        return torch.mm(_load(*_store(s["x"]), K), _load(*s["w"], K).t()).to(dt)
    T, k, D, F = s["T"], s["k"], s["D"], s["F"]
    begin, pairs = s["offsets"].tolist(), s["pairs"].long()
    if op == "experts_glu":
        x = _load(*_store(s["x"]), D)
        h = torch.zeros(T * k, F, dtype=dt, device=x.device)
        for e in range(s["E"]):
            at = pairs[begin[e]:begin[e + 1]]
            if len(at):
                xe = x[at // k]
                g = torch.mm(xe, _load(s["w_gate"][0][e], s["w_gate"][1][e], D).t())
                u = torch.mm(xe, _load(s["w_up"][0][e], s["w_up"][1][e], D).t())
                h[at] = (_gate(g, s["act"]) * u).to(dt)
        return h.reshape(T, k, F)
    h = _load(*_store(s["h"]), F).reshape(T * k, F)
    y = torch.zeros(T * k, D, device=h.device)
    for e in range(s["E"]):
        at = pairs[begin[e]:begin[e + 1]]
        if len(at):
            y[at] = torch.mm(h[at], _load(s["w_down"][0][e], s["w_down"][1][e], F).t())
    return (y.reshape(T, k, D) * s["weights"][:, :, None]).sum(1).to(dt)


def _route_backward(s):
    w, gw = s["weights"].double(), s["grad_weights"].double()
    chosen = s["experts"] >= 0
    at = s["experts"].clamp(min=0).long()
    gw = torch.where(chosen, gw, 0.0)
    score = _scores(s)
    d = torch.zeros_like(score)
    if s["renorm"]:   # w_j = scale s_j / sum s
        gw = gw - (gw * w).sum(-1, keepdim=True) / s["scale"]
    if s["score"] == "sigmoid":
        return d.scatter_add_(1, at, gw * w * (1 - score.gather(1, at)))
    d.scatter_add_(1, at, gw * w)
    return d if s["renorm"] else d - score * (gw * w).sum(-1, keepdim=True)


# ---------------------------------------------------------------------------------------------------- work


def _row(D):   # bytes of a row's codes and scales
    return 17 * -(-D // _BLOCK)


def work(case):
    T, op = case["T"], case["op"]
    if op == "mxfp4":            # x in, codes and scales out; those in, x out
        D = case["D"]
        return {"bytes": 4 * T * D + 2 * T * _row(D), "flops": 4 * T * D}
    if op == "product":
        K, N = case["K"], case["N"]
        return {"bytes": 2 * T * K + N * _row(K) + 2 * T * N, "flops": 2 * T * K * N}
    E, k = case["E"], case["k"]
    if op in ("route", "route_backward"):
        el = T * E * (4 if case["dtype"] == "f32" else 2)
        if op == "route":        # logits in; weights and experts out; the plan out
            return {"bytes": el + (4 * E if case["bias"] else 0) + 8 * T * k + 4 * T * k + 4 * (E + 1), "flops": 8 * T * E}
        every = case["score"] == "softmax" and not case["renorm"]   # else only the chosen logits matter, if any
        some = 0 if case["score"] == "softmax" else el // E * k
        return {"bytes": (el if every else some) + 12 * T * k + el, "flops": (6 if every else 0) * T * E + 8 * T * k}
    D, F = case["D"], case["F"]
    touched = E * (1 - (1 - k / E) ** T)   # experts with a token, of even routing
    if op == "experts_glu":
        return {"bytes": int(2 * T * D + touched * 2 * F * _row(D) + 2 * T * k * F + 4 * T * k), "flops": 4 * T * k * D * F}
    return {"bytes": int(2 * T * k * F + touched * D * _row(F) + 2 * T * D + 8 * T * k), "flops": 2 * T * k * D * F}


# ---------------------------------------------------------------------------------------------------- 64 bits


def _exact_values(x):
    """The values that the 4-bit form of the 16-bit tensor x stands for, from the definition: per run of 32 values the step
    2^e with e the least for which the largest magnitude is under 7 steps (not below 2^-127; 6 steps stay finite in x's format),
    each value the nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6 steps and their negatives, between two the one with an even code."""
    most = 13 if x.dtype == torch.float16 else 125
    d = x.double()
    out = torch.empty_like(d)
    D = x.shape[-1]
    whole = D // _BLOCK * _BLOCK
    for lo, hi in ((0, whole), (whole, D)):
        if hi > lo:
            b = d[..., lo:hi].reshape(*d.shape[:-1], -1, min(_BLOCK, hi - lo))
            top = b.abs().max(-1, keepdim=True).values
            e = torch.floor(torch.log2(top.clamp(min=2.0 ** -140))) - 2
            e = torch.where(top >= 7 * torch.exp2(e), e + 1, e).clamp(min=-127, max=most)
            r = (b / torch.exp2(e)).abs()
            near = torch.zeros_like(r)
            # past the middle of two neighbours the upper one, in the middle the one of even code
            for lower, upper, even in ((0, .5, 0), (.5, 1, 1), (1, 1.5, 0), (1.5, 2, 1), (2, 3, 0), (3, 4, 1), (4, 6, 0)):
                mid = (lower + upper) / 2
                near = torch.where((r >= mid) if even else (r > mid), float(upper), near)
            near = near * torch.exp2(e) * torch.sign(b)
            out[..., lo:hi] = torch.where(torch.isfinite(top), near, torch.nan).reshape(*d.shape[:-1], hi - lo)
    return out


def _exact_load(codes, scales, D):
    c = codes.long()
    c = torch.cat([(c % 16).unsqueeze(-1), (c // 16).unsqueeze(-1)], -1).reshape(*codes.shape[:-1], -1)[..., :D]
    low, mid = c % 2, (c % 8) // 2   # the mantissa bit and the exponent field
    v = torch.where(mid == 0, 0.5 * low, (1 + 0.5 * low) * torch.exp2(mid.double() - 1))
    at = torch.arange(D, device=codes.device) // _BLOCK
    return torch.where(c >= 8, -v, v) * torch.exp2(scales.double() - 127)[..., at]


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "mxfp4":
        return _exact_values(s["x"])
    if op == "product":
        return _exact_values(s["x"]) @ _exact_load(*s["w"], s["K"]).t()
    if op == "route":
        return _route_exact(s)
    if op == "route_backward":
        return _route_backward_exact(s)
    T, k = s["T"], s["k"]
    flat = s["experts"].reshape(-1)
    if op == "experts_glu":
        x = _exact_values(s["x"])
        h = torch.zeros(T * k, s["F"], dtype=torch.float64, device=x.device)
        for e in range(s["E"]):
            at = torch.nonzero(flat == e)[:, 0]
            if at.numel():
                xe = x[at // k]
                g = xe @ _exact_load(s["w_gate"][0][e], s["w_gate"][1][e], s["D"]).t()
                u = xe @ _exact_load(s["w_up"][0][e], s["w_up"][1][e], s["D"]).t()
                if s["act"] == "silu":
                    h[at] = g / (1 + torch.exp(-g)) * u
                else:
                    h[at] = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))) * u
        return h.reshape(T, k, -1)
    h = _exact_values(s["h"]).reshape(T * k, -1)
    y = torch.zeros(T, s["D"], dtype=torch.float64, device=h.device)
    w = s["weights"].double().reshape(-1)
    for e in range(s["E"]):
        at = torch.nonzero(flat == e)[:, 0]
        if at.numel():
            part = h[at] @ _exact_load(s["w_down"][0][e], s["w_down"][1][e], s["F"]).t()
            y.index_add_(0, at // k, part * w[at, None])
    return y


def _exact_scores(s):
    L = s["logits"].double()
    if s["score"] == "sigmoid":
        return torch.sigmoid(L)
    return torch.softmax(L, -1).nan_to_num(0.0)   # a row that is masked throughout has no scores


def _route_exact(s):
    """The definition, an expert (and a group) at a time."""
    T, E, G = s["T"], s["E"], s["groups"]
    score = _exact_scores(s)
    L = s["logits"].double()
    c = L.clone() if s["route_bias"] is None else score + s["route_bias"].double()
    c[L == -math.inf] = -math.inf
    rows = torch.arange(T, device=L.device)
    low = torch.full((T,), -math.inf, dtype=torch.float64, device=L.device)

    def best(v):   # the largest of each row and its first place
        m = v.max(-1).values
        return m, (v == m[:, None]).to(torch.uint8).argmax(-1)

    if G > 1:
        per = E // G
        value = torch.empty(T, G, dtype=torch.float64, device=L.device)
        for i in range(G):
            v = (score if s["route_bias"] is None else c)[:, i * per:(i + 1) * per].clone()
            v[L[:, i * per:(i + 1) * per] == -math.inf] = -math.inf
            first, at = best(v)
            v[rows, at] = low
            second = v.max(-1).values
            value[:, i] = first + second.nan_to_num(neginf=0.0)
        closed = torch.ones(T, G, dtype=torch.bool, device=L.device)
        for _ in range(s["top_groups"]):
            m, at = best(torch.where(closed, value, -math.inf))
            closed[rows, at] = closed[rows, at] & (m == -math.inf)   # no group with an expert is left: none opens
        c[closed.repeat_interleave(per, 1)] = -math.inf
    experts, w = [], []
    for _ in range(s["k"]):
        m, at = best(c)
        none = m == -math.inf
        experts.append(torch.where(none, -1, at))
        w.append(torch.where(none, 0.0, score[rows, at]))
        c[rows, at] = low
    w, experts = torch.stack(w, 1), torch.stack(experts, 1).int()
    if s["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total == 0, 0.0, w / total)
    flat = experts.reshape(-1)
    runs = [torch.nonzero(flat == e)[:, 0] for e in range(E)]
    count = torch.tensor([0] + [len(r) for r in runs], device=L.device)
    return {"weights": w * s["scale"], "experts": experts, "offsets": torch.cumsum(count, 0).int(),
            "pairs": torch.cat(runs + [torch.nonzero(flat < 0)[:, 0]]).int()}


def _route_backward_exact(s):
    """From the scores' Jacobians, with the weights formed again."""
    T, E, k = s["T"], s["E"], s["k"]
    p = _exact_scores(s)
    use = (s["experts"] >= 0).double()
    at = s["experts"].clamp(min=0).long()
    sj = p.gather(1, at) * use
    g = s["grad_weights"].double() * use * s["scale"]
    if s["renorm"]:
        total = sj.sum(1, keepdim=True)
        total = torch.where(total == 0, 1.0, total)
        g = g / total - (g * sj).sum(1, keepdim=True) / total ** 2
    ds = torch.zeros(T, E, dtype=torch.float64, device=p.device)
    for j in range(k):
        ds[torch.arange(T, device=p.device), at[:, j]] += (g * use)[:, j]
    if s["score"] == "sigmoid":
        return ds * p * (1 - p)
    return p * (ds - (ds * p).sum(1, keepdim=True))
