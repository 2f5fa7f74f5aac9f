"""Refusals of the sub-layer's training operators, on the host: the C entry points before any HIP call, and the Python
functions' argument checks before any call into the library."""
import ctypes

import pytest

from mhc_hyper_connection_amd import _binding as B

torch = pytest.importorskip("torch")
import mhc_hyper_connection_amd as mhc

OK, NULL, BAD = B.MHC_OK, B.MHC_ERR_NULLPTR, B.MHC_ERR_PARAM_INVALID
bf, f16, f32 = torch.bfloat16, torch.float16, torch.float32
FAKE = 0x10000   # never dereferenced: every case returns first


def ck(rows, D, dt=0, ptrs=(FAKE, FAKE, FAKE), fn="mhc_checkpoint"):
    p = B.CheckpointParams(rows, D, dt)
    return getattr(B.load(), fn)(ctypes.byref(p), *ptrs, None)


@pytest.mark.parametrize("fn", ["mhc_checkpoint", "mhc_checkpoint_restore"])
def test_checkpoint_refusals(fn):
    for rows, D, dt, want in ((-1, 64, 0, BAD), (4, 0, 0, BAD), (4, 60, 0, BAD), (4, 16392, 0, BAD), (4, 64, 2, BAD), (4, 64, -1, BAD),
                              (1 << 50, 64, 0, BAD), ((1 << 31) * 64, 64, 0, BAD), (0, 64, 1, OK)):
        assert ck(rows, D, dt, fn=fn) == want, (rows, D, dt)
    assert ck(0, 64, ptrs=(None, None, None), fn=fn) == OK
    for i in range(3):
        assert ck(4, 64, ptrs=[None if j == i else FAKE for j in range(3)], fn=fn) == NULL
    first, second = ((FAKE + 8, FAKE, FAKE), (FAKE, FAKE + 8, FAKE))
    assert ck(4, 64, ptrs=first, fn=fn) == BAD
    if fn == "mhc_checkpoint":
        assert ck(4, 64, ptrs=second, fn=fn) == BAD
    else:
        assert ck(4, 64, ptrs=(FAKE, FAKE, FAKE + 8), fn=fn) == BAD
    assert getattr(B.load(), fn)(None, FAKE, FAKE, FAKE, None) == NULL


def post_c(T=4, n=4, D=64, dt=0, res=0, ptrs=(FAKE,) * 5, codes=FAKE, scales=FAKE):
    p, t = B.PostParams(T, n, D, dt, res), B.PostTensors(*ptrs)
    return B.load().mhc_post_checkpoint(ctypes.byref(p), ctypes.byref(t), codes, scales, None)


def test_post_checkpoint_refusals():
    assert post_c(T=-1) == post_c(n=5) == post_c(D=60) == post_c(D=16392) == post_c(dt=2) == post_c(res=1) == post_c(T=1 << 50) == BAD
    assert post_c(T=0, ptrs=(None,) * 5, codes=None, scales=None) == OK
    assert post_c(codes=None) == post_c(scales=None) == post_c(ptrs=(FAKE, None, FAKE, FAKE, FAKE)) == NULL
    assert post_c(codes=FAKE + 8) == post_c(ptrs=(FAKE, FAKE, FAKE + 2, FAKE, FAKE)) == post_c(ptrs=(FAKE + 8, FAKE, FAKE, FAKE, FAKE)) == BAD
    assert B.load().mhc_post_checkpoint(None, None, FAKE, FAKE, None) == NULL


POST_BWD = {f: FAKE for f in B.POST_BWD_TENSOR_FIELDS if f not in ("x_codes", "x_scales", "residual_codes", "residual_scales")}


def post_b(T=4, n=4, D=64, f16_=False, **over):
    return B.raw_post_backward(T, n, D, f16_, {**POST_BWD, **over}, None)


def test_post_backward_refusals():
    assert post_b(T=-1) == post_b(n=3) == post_b(D=4) == post_b(D=16392) == post_b(T=1 << 50) == BAD
    assert B.raw_post_backward(0, 4, 64, False, {}, None) == OK
    for f in POST_BWD:
        assert post_b(**{f: None}) == NULL, f
        assert post_b(**{f: FAKE + 2}) == BAD, f
    assert post_b(x_codes=FAKE) == post_b(x_scales=FAKE) == post_b(residual_codes=FAKE, residual_scales=FAKE) == BAD   # both forms
    assert post_b(x=None, x_codes=FAKE) == post_b(residual=None, residual_scales=FAKE) == NULL                         # half a checkpoint
    assert post_b(x=None, x_codes=FAKE + 8, x_scales=FAKE) == BAD
    assert B.load().mhc_post_backward(None, None, None) == NULL


def pre_b(T=4, n=4, D=64, codes=FAKE, scales=FAKE, ws=FAKE, ws_bytes=1 << 40, num_iters=0, **over):
    ptrs = {f: FAKE for f in B.BWD_TENSOR_FIELDS if f not in ("x", "gamma", "grad_x_post", "grad_gamma")}
    return B.raw_backward_checkpoint(B.make_bwd_params(T, n, D, num_iters=num_iters), {**ptrs, **over}, codes, scales, ws, ws_bytes, None)


def test_pre_backward_checkpoint_refusals():
    assert pre_b(codes=None) == pre_b(scales=None) == pre_b(ws=None) == pre_b(grad_h_in=None) == NULL
    assert pre_b(x=FAKE) == pre_b(codes=FAKE + 8) == pre_b(ws_bytes=16) == pre_b(n=5) == pre_b(D=12) == pre_b(T=-1) == BAD
    assert pre_b(num_iters=2, norm_out=None) == NULL
    assert B.load().mhc_pre_backward_checkpoint(None, None, FAKE, FAKE, FAKE, 1, None) == NULL


def z(*shape, dt=f32):
    return torch.zeros(shape, dtype=dt)


def zck(*shape, dt=bf):
    return mhc.Checkpoint(z(*shape, dt=torch.int8), z(*shape[:-1], -(-shape[-1] // 32), dt=torch.uint8), dt)


def raises(match, fn, *a, **k):
    with pytest.raises(ValueError, match=match):
        fn(*a, **k)


def test_python_checkpoint_checks():
    raises("dtype", mhc.mhc_checkpoint, z(4, 64))
    raises("contiguous", mhc.mhc_checkpoint, z(64, 4, dt=bf).t())
    raises("dimension", mhc.mhc_checkpoint, torch.zeros((), dtype=bf))
    raises("GPU", mhc.mhc_checkpoint, z(4, 64, dt=bf))
    raises("out: a checkpoint of", mhc.mhc_checkpoint, z(4, 64, dt=bf), out=zck(4, 64, dt=f16))
    raises("codes: shape", mhc.mhc_checkpoint, z(4, 64, dt=bf), out=zck(4, 32))
    raises("scales: shape", mhc.mhc_checkpoint, z(4, 72, dt=bf), out=mhc.Checkpoint(z(4, 72, dt=torch.int8), z(4, 2, dt=torch.uint8), bf))
    raises("scales: shape", mhc.mhc_checkpoint_restore, mhc.Checkpoint(z(4, 64, dt=torch.int8), z(4, 1, dt=torch.uint8), bf))
    raises("codes: dtype", mhc.mhc_checkpoint_restore, mhc.Checkpoint(z(4, 64, dt=torch.uint8), z(4, 2, dt=torch.uint8), bf))
    raises("dtype", mhc.mhc_checkpoint_restore, zck(4, 64, dt=f32))
    raises("out: dtype", mhc.mhc_checkpoint_restore, zck(4, 64), out=z(4, 64, dt=f16))
    raises("GPU", mhc.mhc_checkpoint_restore, zck(4, 64))


def test_python_post_checks():
    r, x, p, c = z(3, 4, 64, dt=bf), z(3, 64, dt=bf), z(3, 4), z(3, 4, 4)
    raises("x: dtype", mhc.mhc_post_checkpoint, x.to(f16), r, p, c)
    raises("residual: dtype", mhc.mhc_post_checkpoint, x, r.float(), p, c)
    raises(r"\[T, n, D\]", mhc.mhc_post_checkpoint, x, r[0], p, c)
    raises("comb: shape", mhc.mhc_post_checkpoint, x, r, p, c[:, :3])
    raises("codes: shape", mhc.mhc_post_checkpoint, x, r, p, c, checkpoint=zck(3, 4, 32))
    raises("GPU", mhc.mhc_post_checkpoint, x, r, p, c)
    b = mhc.mhc_post_backward
    raises("x: dtype", b, r, x.to(f16), r, p, c)
    raises("residual: a checkpoint of", b, r, x, zck(3, 4, 64, dt=f16), p, c)
    raises("x.codes: shape", b, r, zck(3, 72), r, p, c)
    raises("x: a tensor or a Checkpoint", b, r, None, r, p, c)
    raises("post: shape", b, r, x, r, z(3, 5), c)
    raises("grad_out: dtype", b, r.float(), x, r, p, c)
    raises(r"\[T, n, D\]", b, r[0], x, r, p, c)
    raises("exactly", b, r, x, r, p, c, out={"grad_x": x})
    raises("GPU", b, r, x, zck(3, 4, 64), p, c)


def test_python_pre_backward_checks():
    n, D, T = 4, 64, 3
    M = n * n + 2 * n
    args = lambda: [z(M, n * D), z(3), z(T, D, dt=bf), z(T, n), z(T, n, n), z(T), z(T, M), z(T, n), z(T, n)]
    r = mhc.PreBackward(T, n, D, device="cpu")
    raises("x: a checkpoint of", r, zck(T, n, D, dt=f16), *args())
    raises("x.codes: shape", r, zck(T, n, D + 8), *args())
    raises("x: a tensor or a Checkpoint", r, None, *args())
    raises("GPU", r, zck(T, n, D), *args())
    raises("multiple of 8", mhc.mhc_pre_backward, zck(T, n, 60), *args())


GLU = dict.fromkeys(("x", "w_gate", "w_up", "h"), FAKE)
GLU_BWD = dict.fromkeys(("grad_h", "x", "w_gate", "w_up", "grad_x", "grad_w_gate", "grad_w_up", "h"), FAKE)


def glu(T=4, D=64, F=128, act=0, dt=0, **over):
    return B.raw_glu(B.GluParams(T, D, F, act, dt), {**GLU, **over}, None)


def glu_b(T=4, D=64, F=128, act=0, dt=0, ws=FAKE, ws_bytes=1 << 50, **over):
    return B.raw_glu_backward(B.GluParams(T, D, F, act, dt), {**GLU_BWD, **over}, ws, ws_bytes, None)


@pytest.mark.parametrize("fn", [glu, glu_b])
def test_glu_refusals(fn):
    for over in (dict(T=-1), dict(T=(1 << 31) + 1), dict(D=0), dict(D=12), dict(D=16392), dict(F=0), dict(F=20), dict(F=65544), dict(act=2),
                 dict(act=-1), dict(dt=2), dict(T=1 << 30, F=65536)):
        assert fn(**over) == BAD, over
    for f in ("x", "w_gate", "w_up", *(("h",) if fn is glu else ("grad_h", "grad_x", "grad_w_gate", "grad_w_up"))):
        assert fn(**{f: None}) == NULL, f
        assert fn(**{f: FAKE + 8}) == BAD, f


def test_glu_backward_forms_and_workspace():
    assert glu_b(x_codes=FAKE) == glu_b(x_scales=FAKE) == BAD                                   # both forms of x
    assert glu_b(x=None, x_codes=FAKE) == glu_b(x=None, x_scales=FAKE) == NULL
    assert glu_b(x=None, x_codes=FAKE + 8, x_scales=FAKE) == glu_b(h=FAKE + 2) == BAD
    assert glu_b(ws=None) == NULL and glu_b(ws=FAKE + 16) == BAD
    p = B.make_glu_params(4, 64, 128, "silu", False)
    need, need_ck = B.glu_backward_workspace_size(p, False), B.glu_backward_workspace_size(p, True)
    assert need >= 4 * 2 * 128 * 2 and need_ck >= need + 4 * 64 * 2
    assert glu_b(ws_bytes=need - 1) == BAD
    assert B.glu_backward_workspace_size(B.make_glu_params(0, 64, 128, "silu", False), True) == 0
    out = ctypes.c_size_t(0)
    size = B.load().mhc_glu_backward_workspace_size
    assert size(None, 0, ctypes.byref(out)) == size(ctypes.byref(p), 0, None) == NULL
    assert size(ctypes.byref(p), 2, ctypes.byref(out)) == BAD
    assert glu(T=0, x=None, h=None) == OK
    assert B.load().mhc_glu(None, None, None) == B.load().mhc_glu_backward(None, None, None, 0, None) == NULL


def test_python_glu_checks():
    x, wg, wu, gh = z(3, 64, dt=bf), z(128, 64, dt=bf), z(128, 64, dt=bf), z(3, 128, dt=bf)
    f, b = mhc.mhc_glu, mhc.mhc_glu_backward
    raises("act", f, x, wg, wu, act="relu")
    raises("x: dtype", f, x.float(), wg, wu)
    raises("w_up: dtype", f, x, wg, wu.to(f16))
    raises("w_up: shape", f, x, wg, wu[:64])
    raises("x: shape", f, z(3, 72, dt=bf), wg, wu)
    raises("w_gate: shape", f, x, wg[0], wu)
    raises("contiguous", f, x, z(64, 128, dt=bf).t(), wu)
    raises("out: shape", f, x, wg, wu, out=z(3, 64, dt=bf))
    raises("GPU", f, x, wg, wu)
    raises("act", b, gh, x, wg, wu, act="")
    raises("grad_h: shape", b, gh[:, :64], x, wg, wu)
    raises("x: dtype", b, gh, x.to(f16), wg, wu)
    raises("x: a checkpoint of", b, gh, zck(3, 64, dt=f16), wg, wu)
    raises("x: a tensor or a Checkpoint", b, gh, None, wg, wu)
    raises("exactly", b, gh, x, wg, wu, out={"grad_x": x})
    raises("exactly", b, gh, x, wg, wu, need_h=True, out={"grad_x": x, "grad_w_gate": wg, "grad_w_up": wu})
    raises("GPU", b, gh, zck(3, 64), wg, wu)


def test_bench_work_matches_the_hand_count():
    import bench
    T, n, D, F = 16384, 4, 7168, 14336
    ck = T * n * (D + 224)
    assert bench.train_work("checkpoint", T, n, D, F) == (2 * T * n * D + ck, 0)
    assert bench.train_work("post_checkpoint", T, n, D, F)[0] == T * (2 * D + 4 * n * D + 4 * n + 4 * n * n) + ck
    assert bench.train_work("post_backward", T, n, D, F)[0] == T * (4 * n * D + 2 * D + D + 224 + 8 * n + 8 * n * n) + ck
    assert bench.train_work("backward_checkpoint", T, n, D, F)[0] == bench.bwd_algorithmic_bytes(T, n, D, num_iters=20) - 2 * T * n * D + ck
    assert bench.train_work("glu", T, n, D, F) == (2 * (T * D + 2 * F * D + T * F), 4 * T * D * F)
    assert bench.train_work("glu_backward", T, n, D, F) == (T * (D + 224) + 8 * F * D + 2 * T * D + 4 * T * F, 12 * T * D * F)


def test_python_pre_backward_checks_the_checkpoint_before_it_reshapes():
    n, D, T = 4, 64, 3
    M = n * n + 2 * n
    args = lambda: [z(M, n * D), z(3), z(T, D, dt=bf), z(T, n), z(T, n, n), z(T), z(T, M), z(T, n), z(T, n)]
    raises("scales: shape", mhc.mhc_pre_backward, mhc.Checkpoint(z(T, n, D, dt=torch.int8), z(T, n, 3, dt=torch.uint8), bf), *args())
    raises("contiguous", mhc.mhc_pre_backward, mhc.Checkpoint(z(T, D, n, dt=torch.int8).transpose(1, 2), z(T, n, 2, dt=torch.uint8), bf), *args())
    raises(r"\[..., n, D\]", mhc.mhc_pre_backward, mhc.Checkpoint(z(D, dt=torch.int8), z(2, dt=torch.uint8), bf), *args())
