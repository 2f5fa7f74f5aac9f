"""Refusals of the routing, the 4-bit floats and the products with 4-bit weights, on the host: the C entry points before any HIP
call, and the Python functions' argument checks before any call into the library. And the launch plans, replayed."""
import ctypes
import os
import subprocess

import pytest

from mhc_hyper_connection_amd import _binding as B

torch = pytest.importorskip("torch")
import mhc_hyper_connection_amd as mhc

OK, NULL, BAD = B.MHC_OK, B.MHC_ERR_NULLPTR, B.MHC_ERR_PARAM_INVALID
bf, f16, f32, i32, u8 = torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.uint8
FAKE = 0x10000   # never dereferenced: every case returns first
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_launch_plans_stay_in_bounds(tmp_path):
    exe = tmp_path / "experts_plan_check"
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "mhc_hyper_connection_amd", "csrc"),
                    os.path.join(ROOT, "tests", "experts_plan_check.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout


def route_p(T=4, E=16, top_k=2, groups=1, top_groups=1, group_top=2, score=0, renormalise=1, dt=2, scale=1.0):
    return B.RouteParams(T, E, top_k, groups, top_groups, group_top, score, renormalise, dt, scale)


def route(ptrs=(FAKE, None, FAKE, FAKE), **kw):
    return B.raw_route(route_p(**kw), *ptrs, None)


def route_b(ptrs=(FAKE,) * 5, **kw):
    return B.raw_route_backward(route_p(**kw), *ptrs, None)


@pytest.mark.parametrize("call", [route, route_b])
def test_route_refusals(call):
    for kw in (dict(T=-1), dict(T=(1 << 26) + 1), dict(E=0), dict(E=1025), dict(top_k=0), dict(top_k=33, E=64), dict(top_k=17), dict(groups=0),
               dict(groups=3), dict(groups=32, E=64), dict(groups=4, top_groups=5), dict(groups=4, top_groups=0),
               dict(groups=4, top_groups=1, top_k=5), dict(group_top=0), dict(group_top=3), dict(score=2), dict(renormalise=2),
               dict(dt=3), dict(dt=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(T=1 << 26, top_k=32, E=64)):
        assert call(**kw) == BAD, kw
    assert call(T=0, ptrs=(None,) * (4 if call is route else 5)) == OK


def test_route_pointers():
    assert route(ptrs=(None, None, FAKE, FAKE)) == route(ptrs=(FAKE, None, None, FAKE)) == route(ptrs=(FAKE, FAKE, FAKE, None)) == NULL
    assert route(ptrs=(FAKE + 2, None, FAKE, FAKE)) == route(ptrs=(FAKE, FAKE + 2, FAKE, FAKE)) == BAD
    assert route(ptrs=(FAKE, None, FAKE + 1, FAKE)) == route(ptrs=(FAKE, None, FAKE, FAKE + 2)) == route(ptrs=(FAKE + 1, None, FAKE, FAKE), dt=0) == BAD
    for i in range(5):
        assert route_b(ptrs=[None if j == i else FAKE for j in range(5)]) == NULL
        assert route_b(ptrs=[FAKE + 2 if j == i else FAKE for j in range(5)]) == BAD
    assert B.load().mhc_route(None, FAKE, None, FAKE, FAKE, None) == B.load().mhc_route_backward(None, *(FAKE,) * 5, None) == NULL


def test_experts_plan_refusals():
    plan = lambda P=64, E=8, ptrs=(FAKE,) * 4, ws=1 << 30: B.raw_experts_plan(P, E, *ptrs, ws, None)
    assert plan(P=-1) == plan(P=1 << 31) == plan(E=0) == plan(E=1025) == BAD
    assert plan(ptrs=(None, FAKE, FAKE, FAKE)) == plan(ptrs=(FAKE, None, FAKE, FAKE)) == plan(ptrs=(FAKE, FAKE, None, FAKE)) == NULL
    assert plan(P=0, ptrs=(None, None, None, None)) == NULL     # the offsets are written even then
    assert plan(P=100000, ptrs=(FAKE, FAKE, FAKE, None)) == NULL
    assert plan(P=100000, ws=16) == plan(P=100000, ptrs=(FAKE, FAKE, FAKE, FAKE + 16)) == plan(ptrs=(FAKE + 2, FAKE, FAKE, FAKE)) == BAD
    assert B.experts_plan_workspace_size(64, 8) == 0
    assert B.experts_plan_workspace_size(100000, 8) == 49 * 9 * 4
    with pytest.raises(mhc.MhcError):
        B.experts_plan_workspace_size(64, 0)
    assert B.load().mhc_experts_plan_workspace_size(64, 8, None) == NULL


@pytest.mark.parametrize("fn", ["mhc_mxfp4", "mhc_mxfp4_restore"])
def test_mxfp4_refusals(fn):
    def call(rows=4, D=64, dt=0, ptrs=(FAKE,) * 3):
        return getattr(B.load(), fn)(ctypes.byref(B.Mxfp4Params(rows, D, dt)), *ptrs, None)
    assert call(rows=-1) == call(D=0) == call(D=65537) == call(dt=2) == call(dt=-1) == call(rows=1 << 50) == call(rows=1 << 28) == BAD
    assert call(rows=0, ptrs=(None,) * 3) == OK
    for i in range(3):
        assert call(ptrs=[None if j == i else FAKE for j in range(3)]) == NULL
        assert call(ptrs=[FAKE + 2 if j == i else FAKE for j in range(3)]) == BAD
    assert getattr(B.load(), fn)(None, FAKE, FAKE, FAKE, None) == NULL


FIELDS = {"mhc_mxfp4_product": (B.ProductTensors, B.PRODUCT_TENSOR_FIELDS, "x", "y"),
          "mhc_experts_glu": (B.ExpertsGluTensors, B.EXPERTS_GLU_TENSOR_FIELDS, "x", "h"),
          "mhc_experts_down": (B.ExpertsDownTensors, B.EXPERTS_DOWN_TENSOR_FIELDS, "h", "y")}


def params(name, **kw):
    if name == "mhc_mxfp4_product":
        return B.Mxfp4ProductParams(*{**dict(T=400, K=4096, N=64, dt=0, reserved=0), **kw}.values())
    return B.ExpertsParams(*{**dict(T=400, E=8, top_k=2, D=4096, F=4096, act=0, dt=0), **kw}.values())


def product(name, ws=FAKE, ws_bytes=1 << 40, p={}, **ptrs):
    cls, fields, left, _ = FIELDS[name]
    t = {f: FAKE for f in fields if f not in (left + "_codes", left + "_scales")}
    t.update(ptrs)
    return B.raw_products(name, params(name, **p), cls(*[t.get(f) for f in fields]), ws, ws_bytes, None)


@pytest.mark.parametrize("name", FIELDS)
def test_products_refusals(name):
    cls, fields, left, out = FIELDS[name]
    bad = [dict(T=-1), dict(dt=2), dict(T=1 << 40)]
    if name == "mhc_mxfp4_product":
        bad += [dict(K=0), dict(K=65537), dict(N=0), dict(N=12), dict(N=65544), dict(reserved=1), dict(T=1 << 30), dict(T=1 << 26, K=32, N=65536)]
    else:
        bad += [dict(E=0), dict(E=1025), dict(top_k=0), dict(top_k=33), dict(D=12), dict(F=12), dict(D=0), dict(F=0), dict(act=2), dict(D=65544),
                dict(F=65544), dict(T=1 << 30, top_k=2)]
    for p in bad:
        assert product(name, p=p) == BAD, p
        with pytest.raises(mhc.MhcError):
            B.products_workspace_size(name, params(name, **p), False)
    codes, scales = left + "_codes", left + "_scales"
    for f in fields:
        if f in (codes, scales):
            continue
        assert product(name, **{f: None}) == NULL, f
        assert product(name, **{f: FAKE + 2}) == BAD, f
    assert product(name, **{codes: FAKE}) == product(name, **{scales: FAKE}) == BAD                # both forms
    assert product(name, **{left: None, codes: FAKE}) == product(name, **{left: None, scales: FAKE}) == NULL
    assert product(name, **{left: None, codes: FAKE + 8, scales: FAKE}) == product(name, **{left: None, codes: FAKE, scales: FAKE + 2}) == BAD
    assert product(name, ws=None) == NULL
    assert product(name, ws=FAKE + 16) == product(name, ws_bytes=64) == BAD
    assert product(name, p=dict(T=0), ws=None, **{f: None for f in fields if not f.startswith("w_")}) == OK
    assert B.raw_products(name, params(name), cls(), None, 0, None) == NULL
    lib = B.load()
    assert getattr(lib, name)(None, None, None, 0, None) == NULL
    size = ctypes.c_size_t(0)
    get = getattr(lib, name + "_workspace_size")
    assert get(None, 0, ctypes.byref(size)) == get(ctypes.byref(params(name)), 0, None) == NULL
    assert get(ctypes.byref(params(name)), 2, ctypes.byref(size)) == BAD
    assert B.products_workspace_size(name, params(name), False) > 0
    few = params(name, T=1)                   # the streaming kernel rounds x itself
    assert (B.products_workspace_size(name, few, False) > 0) == (name == "mhc_experts_down")
    assert (B.products_workspace_size(name, params(name), True) > 0) == (name == "mhc_experts_down")


def test_the_weighted_sums_grid_is_bounded():
    assert product("mhc_experts_down", p=dict(T=1 << 20, top_k=32, F=64, D=16384)) == BAD


def z(*shape, dt=bf):
    return torch.zeros(shape, dtype=dt)


def m4(*shape, dt=bf):
    D = shape[-1]
    return mhc.Mxfp4(z(*shape[:-1], 16 * -(-D // 32), dt=u8), z(*shape[:-1], 4 * -(-D // 128), dt=u8), dt, D)


def refused(match, f, *a, **k):
    with pytest.raises(ValueError, match=match):
        f(*a, **k)


def test_python_route_checks():
    r = mhc.mhc_route
    L = z(4, 16, dt=f32)
    refused("logits: dtype", r, z(4, 16, dt=torch.float64), 2)
    refused("score", r, L, 2, score="relu")
    refused("top_k", r, L, 0)
    refused("contiguous", r, z(16, 4, dt=f32).t(), 2)
    refused("bias: shape", r, L, 2, bias=z(8, dt=f32))
    refused("bias: dtype", r, L, 2, bias=z(16))
    refused("at least one dimension", r, torch.zeros(()), 1)
    refused(r"out\[0\]: shape", r, L, 2, out=(z(4, 3, dt=f32), z(4, 2, dt=i32)))
    refused(r"out\[1\]: dtype", r, L, 2, out=(z(4, 2, dt=f32), z(4, 2, dt=torch.int64)))
    refused(r"out\[1\] is required", r, L, 2, out=(z(4, 2, dt=f32), None))
    refused("on a GPU", r, L, 2)
    b = mhc.mhc_route_backward
    w, e = z(4, 2, dt=f32), z(4, 2, dt=i32)
    refused("grad_weights: dtype", b, z(4, 2), L, w, e)
    refused("grad_weights is required", b, None, L, w, e)
    refused("weights: shape", b, w, L, z(4, 3, dt=f32), e)
    refused("experts: dtype", b, w, L, w, w)
    refused("out: dtype", b, w, L, w, e, out=z(4, 16))
    refused("on a GPU", b, w, L, w, e)
    refused("experts: dtype", mhc.mhc_experts_plan, w, 16)
    refused("contiguous", mhc.mhc_experts_plan, z(2, 4, dt=i32).t(), 16)
    refused("on a GPU", mhc.mhc_experts_plan, e, 16)


def test_python_mxfp4_checks():
    q, s = mhc.mhc_mxfp4, mhc.mhc_mxfp4_restore
    refused("x: dtype", q, z(4, 64, dt=f32))
    refused("contiguous", q, z(64, 4).t())
    refused("at least one dimension", q, torch.zeros((), dtype=bf))
    refused("out: an Mxfp4", q, z(4, 64), out=z(4, 64))
    refused("out: of 32 values", q, z(4, 64), out=m4(4, 32))
    refused("out.codes: shape", q, z(4, 64), out=m4(5, 64))
    refused("out: of dtype", q, z(4, 64), out=m4(4, 64, dt=f16))
    refused("on a GPU", q, z(4, 64))
    refused("m: of dtype", s, m4(4, 64)._replace(dtype=f32))
    refused("m.scales: shape", s, m4(4, 64)._replace(scales=z(4, 2, dt=u8)))
    refused("m.codes: shape", s, m4(4, 64)._replace(size=65))
    refused("out: shape", s, m4(4, 64), out=z(4, 63))
    refused("on a GPU", s, m4(4, 64))


def test_python_products_checks():
    p, g, d = mhc.mhc_mxfp4_product, mhc.mhc_experts_glu, mhc.mhc_experts_down
    refused("x: dtype", p, z(4, 64, dt=f32), m4(8, 64))
    refused("w: an Mxfp4", p, z(4, 64), z(8, 64))
    refused("w: an Mxfp4", p, z(4, 64), m4(2, 8, 64))
    refused("w: of 32 values", p, z(4, 64), m4(8, 32))
    refused("out: shape", p, z(4, 64), m4(8, 64), out=z(4, 16))
    refused("out: dtype", p, z(4, 64), m4(8, 64), out=z(4, 8, dt=f16))
    refused("on a GPU", p, m4(4, 64), m4(8, 64))
    plan = mhc.ExpertsPlan(z(9, dt=i32), z(8, dt=i32), (4, 2))
    x, w = z(4, 64), m4(8, 16, 64)
    refused("act", g, x, plan, w, w, act="relu")
    refused("w_gate: an Mxfp4", g, x, plan, m4(16, 64), w)
    refused("w_up.codes: shape", g, x, plan, w, m4(8, 24, 64))
    refused("plan: an ExpertsPlan", g, x, None, w, w)
    refused("plan.offsets: shape", g, x, plan._replace(offsets=z(8, dt=i32)), w, w)
    refused("plan.pairs: dtype", g, x, plan._replace(pairs=z(8, dt=torch.int64)), w, w)
    refused("plan: of shape", g, z(8, 64), plan, w, w)
    refused("plan.pairs: shape", g, x, plan._replace(shape=(4, 3)), w, w)
    refused("out: shape", g, x, plan, w, w, out=z(4, 2, 8))
    refused("on a GPU", g, x, plan, w, w)
    h, wd, ws = z(4, 2, 64), m4(8, 16, 64), z(4, 2, dt=f32)
    refused("w_down: an Mxfp4", d, h, plan, ws, m4(16, 64))
    refused("plan: of shape", d, z(8, 64), plan, ws, wd)
    refused("weights is required", d, h, plan, None, wd)
    refused("weights: dtype", d, h, plan, z(4, 2), wd)
    refused("out: shape", d, h, plan, ws, wd, out=z(4, 2, 16))
    refused("on a GPU", d, h, plan, ws, wd)
