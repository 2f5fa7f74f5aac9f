"""The gated projection and its backward over every tile shape, format and activation, sharply.

Whole numbers: inputs whose products and sums are whole numbers below 2^24, with gates so far out that act(g) is g or 0 and
act'(g) 1 or 0 to the last bit. Every fp32 sum is then exact in whatever order, dg and du too, and each result is the whole number's
one rounding: equal bit for bit, no tolerance.

Random values, dg and du read from the workspace ([dg | du], as include/mhc.h has it): they are held against the formula in 64
bits as tests/test_gpu_glu.py does, and the results against the 64-bit products of the dg and du that were read, so that only
the results' own fp32 sums and one rounding are left. A matrix instruction adds 32 products to the sum so far, at most 32
additions, each off by at most u = 2^-24 of what it has seen: 32 u (|sum| + the products' magnitudes). Over S = K / 32
instructions the magnitudes add up to A, and the sums so far to S times their largest, taken as 5 R with R^2 the sum of the
squares of all K products (partial sums of terms of random sign: five standard deviations). The parts of a cut tile, at most
43 here, add as many additions of such sums. So a result is off by 32 u (5 S R + A) + 43 u 5 R, and then half a step."""
import sys

import pytest

from gpu_helpers import device
from test_gpu_glu import FN, U, act_ref
from train_helpers import torch_dtype

pytestmark = pytest.mark.gpu

# few tokens; 128 x 128 tiles, whole and cut; 256 x 256 tiles of all three products, whole and cut in 2 to 43 parts, alone and
# beside whole ones, with partial tiles along T, D and F
SIZES = [(1, 264, 1000), (17, 96, 2048), (33, 40, 264), (64, 1032, 264), (40, 1032, 8200), (65, 4104, 200), (300, 2048, 544), (1003, 2048, 5464), (1030, 2560, 4104),
         (4099, 1032, 2056), (4099, 4104, 520), (513, 4104, 1032), (2049, 520, 4104)]


def whole_inputs(T, D, F, dtype, seed):
    import torch
    g = torch.Generator(device=device()).manual_seed(seed)
    some = lambda *s, p, top=1: torch.where(torch.rand(s, generator=g, device=device()) < p, torch.randint(-top, top + 1, s, generator=g, device=device()).float(), 0.0)
    x, wg, wu = some(T, D, p=0.1), some(F, D, p=0.1), some(F, D, p=0.1, top=2)
    x[:, 0] = 16.0
    wg[:, 0] = torch.where(torch.rand(F, generator=g, device=device()) < 0.25, -16.0, 8.0)   # a quarter of the gates shut: g about -256
    wu[:, 0] = 0.0
    gh = torch.randint(-3, 4, (T, F), generator=g, device=device()).float()
    return {k: v.to(dtype) for k, v in dict(x=x, w_gate=wg, w_up=wu, grad_h=gh).items()}


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("T,D,F", SIZES)
def test_whole_numbers_are_exact(T, D, F, f16, act):
    import mhc_hyper_connection_amd as mhc
    import torch
    dt = torch_dtype(f16)
    print(f"[case] glu whole numbers T={T} D={D} F={F} f16={f16} {act}", file=sys.stderr, flush=True)
    d = whole_inputs(T, D, F, dt, seed=T + D + F)
    x, wg, wu, gh = (d[k].double() for k in ("x", "w_gate", "w_up", "grad_h"))
    g, u = x @ wg.t(), x @ wu.t()
    a, da = torch.where(g > 0, g, torch.zeros_like(g)), (g > 0).double()
    assert float(g.abs().min()) >= 64                       # e^-64 is nothing beside 1 in fp32
    dg, du = gh * u * da, gh * a
    assert float(max(dg.abs().max(), du.abs().max())) < 2 ** 11      # one rounding, none in fp16
    dg, du = dg.to(dt).double(), du.to(dt).double()
    exact = {"h": a * u, "grad_x": dg @ wg + du @ wu, "grad_w_gate": dg.t() @ x, "grad_w_up": du.t() @ x}
    for A in (dg.abs() @ wg.abs() + du.abs() @ wu.abs(), dg.abs().t() @ x.abs(), du.abs().t() @ x.abs()):
        assert float(A.max()) < 2 ** 24
    want = {k: v.to(torch.float32).to(dt) for k, v in exact.items()}
    got = {"fwd": mhc.mhc_glu(d["x"], d["w_gate"], d["w_up"], act=act)}
    assert torch.equal(got["fwd"], want["h"])
    for kept in (False, True):
        xk = mhc.mhc_checkpoint(d["x"]) if kept else d["x"]
        if kept:
            assert torch.equal(mhc.mhc_checkpoint_restore(xk), d["x"])
        full = {k: torch.full((v.shape[0] + 1, v.shape[1]), 7.0, dtype=dt, device=v.device) for k, v in want.items()}
        out = mhc.mhc_glu_backward(d["grad_h"], xk, d["w_gate"], d["w_up"], act=act, need_h=True, out={k: v[:-1] for k, v in full.items()})
        for k in want:
            assert torch.equal(out[k], want[k]), (k, kept, int((out[k] != want[k]).sum()))
            assert (full[k][-1] == 7.0).all(), k


def random_inputs(T, D, F, dtype, seed, grad):
    import torch
    g = torch.Generator(device=device()).manual_seed(seed)
    f = lambda *s, std=1.0: (std * torch.randn(*s, generator=g, device=device())).to(dtype)
    return dict(x=f(T, D), w_gate=f(F, D, std=2 / D ** 0.5), w_up=f(F, D, std=1 / D ** 0.5), grad_h=f(T, F, std=grad))


def backward_with_workspace(d, x, act, kept):
    """mhc_glu_backward's outputs, and dg and du as its workspace holds them."""
    import mhc_hyper_connection_amd as mhc
    import torch
    dev, dt = device(), d["grad_h"].dtype
    T, F = d["grad_h"].shape
    D = d["w_gate"].shape[1]
    p = mhc.make_glu_params(T, D, F, act, dt == torch.float16)
    size = mhc.glu_backward_workspace_size(p, kept)
    ws = torch.empty(size, dtype=torch.uint8, device=dev)
    out = dict(grad_x=torch.empty((T, D), dtype=dt, device=dev), grad_w_gate=torch.empty((F, D), dtype=dt, device=dev),
               grad_w_up=torch.empty((F, D), dtype=dt, device=dev), h=torch.empty((T, F), dtype=dt, device=dev))
    ptrs = {**{k: d[k].data_ptr() for k in ("grad_h", "w_gate", "w_up")}, **{k: v.data_ptr() for k, v in out.items()}}
    if kept:
        ptrs.update(x_codes=x.codes.data_ptr(), x_scales=x.scales.data_ptr())
    else:
        ptrs["x"] = x.data_ptr()
    assert mhc.raw_glu_backward(p, ptrs, ws.data_ptr(), size, torch.cuda.current_stream(dev).cuda_stream) == mhc.MHC_OK
    dgu = ws[:T * 2 * F * 2].view(dt).view(T, 2 * F)
    return out, dgu[:, :F].clone(), dgu[:, F:].clone()


def half(ref, f16):
    """train_helpers.half_step on the GPU."""
    eps, least = (2.0 ** -11, 2.0 ** -25) if f16 else (2.0 ** -8, 2.0 ** -134)
    return (eps * ref.abs()).clamp(min=least)


CASES = [(1003, 2048, 5464, True, "gelu_tanh", 1.0, True), (1003, 2048, 5464, True, "silu", 1e-4, False), (1003, 2048, 5464, True, "silu", 1e3, True),
         (1030, 2560, 4104, False, "gelu_tanh", 1.0, True), (4099, 1032, 2056, True, "gelu_tanh", 1e-4, False), (513, 4104, 1032, False, "silu", 1e-4, True),
         (300, 2048, 544, True, "silu", 1e-4, True), (20, 2048, 544, True, "gelu_tanh", 1e-4, False), (20, 2048, 544, True, "silu", 1e3, False),
         (4099, 1032, 2056, True, "silu", 1.0, False), (513, 4104, 1032, False, "silu", 1.0, True), (300, 2048, 544, True, "silu", 1.0, True),
         (20, 2048, 544, True, "gelu_tanh", 1.0, False)]


@pytest.mark.parametrize("T,D,F,f16,act,grad,kept", CASES)
def test_results_from_the_dg_and_du_that_are_held(T, D, F, f16, act, grad, kept):
    import mhc_hyper_connection_amd as mhc
    import torch
    print(f"[case] glu random T={T} D={D} F={F} f16={f16} {act} grad={grad} kept={kept}", file=sys.stderr, flush=True)
    d = random_inputs(T, D, F, torch_dtype(f16), seed=T + F, grad=grad)
    xk = mhc.mhc_checkpoint(d["x"]) if kept else d["x"]
    x = mhc.mhc_checkpoint_restore(xk).double() if kept else d["x"].double()
    out, dg, du = backward_with_workspace(d, xk, act, kept)
    wg, wu, gh = (d[k].double() for k in ("w_gate", "w_up", "grad_h"))
    g, u = x @ wg.t(), x @ wu.t()
    eg, eu = D * U * (x.abs() @ wg.abs().t()), D * U * (x.abs() @ wu.abs().t())
    a, da = (torch.from_numpy(t).to(g.device) for t in act_ref(g.cpu().numpy(), act))

    def holds(name, got, want, lim):
        lim = lim + half(want.abs() + lim, f16)
        bad = ~((got.double() - want).abs() <= lim)
        if f16:   # 65520 and more rounds to fp16's infinity: 65504 + half a step of 32
            bad &= ~(torch.isinf(got) & (got.double() * want > 0) & (want.abs() + lim >= 65520.0))
        assert not bad.any(), (name, int(bad.sum()), float(((got.double() - want).abs() / lim)[bad].max()))

    holds("h", out["h"], a * u, 1.13 * eg * u.abs() + a.abs() * eu + FN * (a * u).abs())
    holds("dg", dg, gh * u * da, gh.abs() * (1.13 * eu + 0.8 * eg * u.abs()) + FN * (gh * u).abs())
    holds("du", du, gh * a, gh.abs() * 1.13 * eg + FN * (gh * a).abs())
    dg, du = dg.double(), du.double()
    assert torch.isfinite(dg).all() and torch.isfinite(du).all()

    def product(name, terms, K):
        want, A, R = sum(p @ q for p, q in terms), sum(p.abs() @ q.abs() for p, q in terms), sum(p.square() @ q.square() for p, q in terms).sqrt()
        holds(name, out[name], want, 32 * U * (5 * (K / 32) * R + A) + 43 * U * 5 * R)

    product("grad_x", ((dg, wg), (du, wu)), 2 * F)
    product("grad_w_gate", ((dg.t(), x),), T)
    product("grad_w_up", ((du.t(), x),), T)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("T,D,F", [(1, 264, 1000), (16, 512, 136), (17, 96, 2048), (32, 72, 4104), (33, 2056, 264), (64, 128, 1032), (65, 72, 40), (300, 2048, 544),
                                   (1003, 2048, 5464)])
def test_h_again_is_the_forwards_h(T, D, F, f16, act):
    # one kernel computes h in both directions, for few tokens as for many: the same bits
    import mhc_hyper_connection_amd as mhc
    import torch
    print(f"[case] glu h again T={T} D={D} F={F} f16={f16} {act}", file=sys.stderr, flush=True)
    d = random_inputs(T, D, F, torch_dtype(f16), seed=T, grad=1.0)
    h = mhc.mhc_glu(d["x"], d["w_gate"], d["w_up"], act=act)
    got = mhc.mhc_glu_backward(d["grad_h"], d["x"], d["w_gate"], d["w_up"], act=act, need_h=True)
    assert torch.equal(got["h"].view(torch.int16), h.view(torch.int16))


@pytest.mark.parametrize("T,D,F", [(20, 264, 136), (300, 264, 136), (1003, 2048, 5464)])
def test_fp16_range_of_dg_and_du(T, D, F):
    # dg and du are fp16 tensors. A grad_h of 60000 leaves their range wherever act(g) or u act'(g) passes 1.1, as it does for some f
    # of any token here: that token's grad_x is not finite, and no other token's changes. The same gradients 2^-14
    # times the size (a smaller loss scale) are in range.
    import mhc_hyper_connection_amd as mhc
    import torch
    print(f"[case] glu fp16 range T={T} D={D} F={F}", file=sys.stderr, flush=True)
    d = random_inputs(T, D, F, torch.float16, seed=7, grad=1.0)
    t = T // 2
    keep = [k for k in range(T) if k != t]
    base = mhc.mhc_glu_backward(d["grad_h"], d["x"], d["w_gate"], d["w_up"])
    d["grad_h"][t] = 60000.0
    big = mhc.mhc_glu_backward(d["grad_h"], d["x"], d["w_gate"], d["w_up"])
    assert torch.equal(big["grad_x"][keep], base["grad_x"][keep])
    assert not torch.isfinite(big["grad_x"][t]).all()
    d["grad_h"][t] *= 2.0 ** -14
    small = mhc.mhc_glu_backward(d["grad_h"], d["x"], d["w_gate"], d["w_up"])
    assert all(torch.isfinite(v).all() for v in small.values())
