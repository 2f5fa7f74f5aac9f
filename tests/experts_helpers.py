"""References of the routing to experts, the microscaled 4-bit floats and the products with 4-bit weights, in 64 bits on the
CPU, written from the definitions in include/mhc.h."""
import numpy as np

from train_helpers import half_step, to_16, torch_dtype   # noqa: F401

U = 2.0 ** -24
VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def quantise(v, f16):
    """Codes uint8 [..., D] (one to a byte, sign in bit 3) and scale bytes [..., ceil(D / 32)] of the float64 array v of
    16-bit values, from the definition: the least step 2^e with the block's largest magnitude under 7 steps."""
    lead, D = v.shape[:-1], v.shape[-1]
    nb = -(-D // 32)
    b = np.zeros((*lead, nb * 32))
    b[..., :D] = v
    b = b.reshape(*lead, nb, 32)
    bad = ~np.isfinite(b).all(-1)
    neg = np.signbit(b)
    b = np.abs(np.where(bad[..., None], 0.0, b))
    top = b.max(-1)
    e = np.full(top.shape, -127)
    for x in range(-127, 126):                       # the least e that fits
        e = np.where(top >= 7 * np.ldexp(1.0, x), x + 1, e)
    e = np.minimum(e, 13 if f16 else 125)
    r = np.ldexp(b, -e[..., None])
    # the nearest of the eight values, ties to the even code
    d = np.abs(r[..., None] - VALUES)
    near = d.min(-1, keepdims=True)
    tied = d == near
    first = tied.argmax(-1)
    c = np.where((tied.sum(-1) == 2) & (first % 2 == 1), first + 1, first)
    c = np.where(bad[..., None], 0, c + 8 * neg)
    s = np.where(bad, 255, e + 127)
    return c.reshape(*lead, nb * 32).astype(np.uint8), s.astype(np.uint8)


def pack(c, s):
    """The library's layout of codes (one to a byte, whole blocks) and scale bytes."""
    nb = s.shape[-1]
    codes = (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)
    scales = np.zeros((*s.shape[:-1], 4 * -(-nb // 4)), np.uint8)
    scales[..., :nb] = s
    return codes, scales


def values(codes, scales, D):
    """What packed codes and scales stand for, in float64."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)[..., :D]
    v = np.where(c >= 8, -1.0, 1.0) * VALUES[c & 7]
    s = scales.astype(np.int64)
    step = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return v * np.repeat(step, 32, -1)[..., :D]


def rounded(v, f16):
    """The 4-bit values of 16-bit values."""
    c, s = quantise(v, f16)
    return values(*pack(c, s), v.shape[-1])


def mxfp4(rng, *shape, low=124, high=130):
    """Random codes and scales of [.., D], packed, as numpy arrays; the padding zero."""
    D = shape[-1]
    nb = -(-D // 32)
    c = rng.integers(0, 16, (*shape[:-1], nb * 32)).astype(np.uint8)
    c[..., D:] = 0
    s = rng.integers(low, high, (*shape[:-1], nb)).astype(np.uint8)
    return pack(c, s)


def to_mxfp4(codes, scales, D, f16, dev):
    import mhc_hyper_connection_amd as mhc
    import torch
    return mhc.Mxfp4(torch.from_numpy(np.ascontiguousarray(codes)).to(dev), torch.from_numpy(np.ascontiguousarray(scales)).to(dev),
                     torch_dtype(f16), D)


def scores(L, score):
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1 / (1 + np.exp(-L))
        top = L.max(-1, keepdims=True)
        p = np.exp(L - np.where(np.isfinite(top), top, 0))
        p = np.where(top == np.inf, np.nan, p)
        total = p.sum(-1, keepdims=True)
        return p / np.where(total == 0, 1, total)


def route(L, k, bias=None, score="softmax", groups=1, top_groups=1, group_top=2, renormalise=True, scale=1.0):
    """weights, experts of float64 logits [T, E], a token at a time."""
    T, E = L.shape
    s = scores(L, score)
    weights, experts = np.zeros((T, k)), np.full((T, k), -1, np.int32)
    for t in range(T):
        b = np.zeros(E) if bias is None else bias
        if np.isnan(L[t]).any() or np.isnan(b).any() or (score == "softmax" and (L[t] == np.inf).any()):
            weights[t] = np.nan
            continue
        allowed = [e for e in range(E) if L[t, e] != -np.inf and b[e] != -np.inf]
        c = s[t] + b
        if groups > 1:
            per = E // groups
            value = {}
            for g in range(groups):
                best = sorted((c[e] for e in allowed if e // per == g), reverse=True)[:group_top]
                if best:
                    value[g] = sum(best)
            stay = sorted(value, key=lambda g: (-value[g], g))[:top_groups]
            allowed = [e for e in allowed if e // per in stay]
        key = L[t] if bias is None else c
        chosen = sorted(allowed, key=lambda e: (-key[e], e))[:k]
        w = s[t][chosen]
        if renormalise and w.sum() > 0:
            w = w / w.sum()
        weights[t, :len(chosen)], experts[t, :len(chosen)] = w * scale, chosen
    return weights, experts


def route_backward(gw, L, weights, experts, score="softmax", renormalise=True, scale=1.0):
    """(gradient, bound of the error before the last rounding), from the formulas, with the weights that were given."""
    T, E = L.shape
    s = scores(L, score)
    use = (experts >= 0) & (experts < E)
    at = np.where(use, experts, 0)
    rows = np.arange(T)[:, None]
    g, w = np.where(use, gw, 0), np.where(use, weights, 0)
    S = (g * (w / scale)).sum(1, keepdims=True)
    d = w * (g - S if renormalise else g)
    if score == "sigmoid":
        d = np.where(use, d * scores(-L, score)[rows, at], 0)     # 1 - s is the sigmoid of -l, without cancelling
    out, lim = np.zeros((T, E)), np.zeros((T, E))
    np.add.at(out, (rows, at), np.where(use, d, 0))
    if score == "softmax" and not renormalise:
        # fp32: the chosen's term, and s_e S scale, whose exponent's argument, sum of E terms and three products are rounded
        lim += U * np.abs(out)
        with np.errstate(invalid="ignore"):
            far = np.where(np.isfinite(L), L.max(-1, keepdims=True) - L, 0).max(-1, keepdims=True)
        sub = s * S * scale
        lim += np.abs(sub) * U * (2 * far + 40)
        # under 2^-126 fp32's steps are 2^-149 whatever the value: the exponential is off by one of them, which S scale (over a
        # sum of at least 1) multiplies, and the product by half of one
        lim += 2.0 ** -149 * (np.abs(S * scale) + 0.5)
        out = out - sub
    bad = np.isnan(weights).any(1)
    out[bad] = np.nan
    return out, lim


def plan(experts, E):
    flat = experts.reshape(-1)
    e = np.where((flat < 0) | (flat >= E), E, flat)
    pairs = np.argsort(e, kind="stable").astype(np.int32)
    offsets = np.searchsorted(e[pairs], np.arange(E + 1)).astype(np.int32)
    return offsets, pairs


def act_ref(g, act):
    with np.errstate(over="ignore"):
        z = g if act == "silu" else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
        return g / (1 + np.exp(-z))


def sum_error(K, magnitude):
    """Of an fp32 sum of K exact products whose magnitudes add up to `magnitude`: the matrix instruction adds 128 at a time, each
    of which may be cut at fp32's last bit of the largest, then ceil(K / 128) partial sums are rounded, and four waves' joined."""
    return U * (2 * 128 + -(-K // 128) + 8) * magnitude


def check(name, got, want, lim, f16):
    """Every value within lim and one rounding to 16 bits; NaN where wanted."""
    got = got.double().cpu().numpy() if not isinstance(got, np.ndarray) else got
    assert got.shape == want.shape, name
    assert (np.isnan(got) == np.isnan(want)).all(), (name, "NaN")
    ok = ~np.isnan(want)
    if f16:   # past the largest value comes infinity
        top = 65504.0
        want = np.where(np.abs(want) >= 65520, np.copysign(np.inf, want), want)
        over = np.isinf(want) | (np.abs(want) + lim >= top)
        ok &= ~over
        assert ((np.abs(got[over]) >= top - lim[over])).all(), (name, "range")
    lim = lim + half_step(np.abs(want) + lim, f16)
    err = np.abs(got[ok] - want[ok])
    assert (err <= lim[ok]).all(), (name, float((err / lim[ok]).max()), int((~(err <= lim[ok])).sum()))
