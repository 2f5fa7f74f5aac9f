"""Microscaled 4-bit floats on the GPU: codes, scale bytes and restored values equal the definition's, bit for bit."""
import sys

import numpy as np
import pytest

from experts_helpers import pack, quantise, to_16, torch_dtype, values
from gpu_helpers import device

pytestmark = pytest.mark.gpu


def check(x, f16, dev):
    """x: a 16-bit torch CPU tensor [.., D]"""
    import mhc_hyper_connection_amd as mhc
    import torch
    v, D = x.double().numpy(), x.shape[-1]
    m = mhc.mhc_mxfp4(x.to(dev))
    codes, scales = pack(*quantise(v, f16))
    assert m.size == D and m.dtype == x.dtype
    assert np.array_equal(m.scales.cpu().numpy(), scales)
    got = m.codes.cpu().numpy()
    assert np.array_equal(got, codes), np.argwhere(got != codes)[:4].tolist()
    want = values(codes, scales, D)
    back = mhc.mhc_mxfp4_restore(m)
    assert back.dtype == x.dtype and back.shape == x.shape
    assert np.array_equal(back.double().cpu().numpy(), want, equal_nan=True)
    # twice in 4 bits is once: the values that come back are exact
    again = mhc.mhc_mxfp4_restore(mhc.mhc_mxfp4(back))
    finite = torch.from_numpy(np.isfinite(want).reshape(-1, D).all(-1))
    assert torch.equal(again.cpu().reshape(-1, D)[finite], back.cpu().reshape(-1, D)[finite])
    return v, want


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (1, 8), (5, 24), (2, 31), (4, 32), (3, 33), (7, 40), (2, 64), (9, 100), (3, 128), (5, 136), (4, 250), (2, 3, 256),
                                   (1003, 72), (130, 1000), (65, 2048), (33, 5464), (7,), (300, 401)])
def test_sizes(shape, f16):
    print(f"[case] mxfp4 {shape} f16={f16}", file=sys.stderr, flush=True)
    rng = np.random.default_rng(sum(shape))
    x = to_16(rng.standard_normal(shape) * np.exp(2 * rng.standard_normal((*shape[:-1], 1))), f16)
    v, want = check(x, f16, device())
    D = shape[-1]
    b = np.pad(np.abs(v), [(0, 0)] * (v.ndim - 1) + [(0, -D % 32)]).reshape(*shape[:-1], -1, 32).max(-1)
    # the documented bound
    assert (np.abs(want - v) <= np.repeat(b, 32, -1)[..., :D] / 5 * (1 + 1e-12) + 2.0 ** -129).all()


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("D", [32, 128, 40])
def test_every_value(D, f16):
    # every 16-bit value: beside its neighbours, beside others, and as its block's largest
    import torch
    dev = device()
    bits = np.arange(65536, dtype=np.uint16)
    rng = np.random.default_rng(1)
    for kind in range(3):
        print(f"[case] every value D={D} f16={f16} kind={kind}", file=sys.stderr, flush=True)
        if kind == 0:
            rows = bits[:65536 // D * D].reshape(-1, D)
        elif kind == 1:
            rows = rng.permutation(bits)[:65536 // D * D].reshape(-1, D)
        else:
            rows = np.zeros((65536, D), np.uint16)
            rows[:, D // 3] = bits
            rows[:, D // 3 + 1] = bits // 2          # a smaller one
        check(torch.from_numpy(rows.view(np.int16).copy()).view(torch_dtype(f16)), f16, dev)


@pytest.mark.parametrize("f16", [False, True])
def test_every_code_and_scale(f16):
    # restored values of every pair of codes and every scale byte
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    codes = np.tile(np.arange(256, dtype=np.uint8).reshape(16, 16), (256, 1))           # 16 rows of one block for each scale
    scales = np.zeros((4096, 4), np.uint8)
    scales[:, 0] = np.repeat(np.arange(256), 16)
    m = mhc.Mxfp4(torch.from_numpy(codes).to(dev), torch.from_numpy(scales).to(dev), torch_dtype(f16), 32)
    got = mhc.mhc_mxfp4_restore(m).double().cpu().numpy()
    v = values(codes, scales, 32)
    with np.errstate(over="ignore"):                                                      # past fp32's range, at 254
        finite = torch.from_numpy(np.nan_to_num(v).astype(np.float32))
    want = finite.to(torch_dtype(f16)).double().numpy()
    want[np.isnan(v)] = np.nan
    assert np.array_equal(got, want, equal_nan=True)


def test_rows_past_32_bits():
    # offsets of x past 2^32 bytes: the last rows
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    for D in (8192, 8200):
        rows = (1 << 32) // (2 * D) + 300
        print(f"[case] mxfp4 rows={rows} D={D}", file=sys.stderr, flush=True)
        x = torch.zeros((rows, D), dtype=torch.bfloat16, device=dev)
        tail = torch.randn((200, D), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
        x[-200:] = tail.to(dev)
        m = mhc.mhc_mxfp4(x)
        few = mhc.mhc_mxfp4(tail.to(dev))
        assert torch.equal(m.codes[-200:], few.codes) and torch.equal(m.scales[-200:], few.scales)
        assert (m.codes[:-200] == 0).all()
        back = mhc.mhc_mxfp4_restore(m, out=x)
        assert torch.equal(back[-200:], mhc.mhc_mxfp4_restore(few))
        assert (back[:-200] == 0).all()
        del x, m, back


def test_outputs_given_and_empty():
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    x = torch.randn(6, 100, device=dev).to(torch.bfloat16)
    full = mhc.Mxfp4(torch.full((7, 64), 7, dtype=torch.uint8, device=dev), torch.full((7, 4), 7, dtype=torch.uint8, device=dev), torch.bfloat16, 100)
    out = full._replace(codes=full.codes[:6], scales=full.scales[:6])
    assert mhc.mhc_mxfp4(x, out=out) is out
    want = mhc.mhc_mxfp4(x)
    assert torch.equal(out.codes, want.codes) and torch.equal(out.scales, want.scales)
    assert (full.codes[6] == 7).all() and (full.scales[6] == 7).all()
    back = torch.full((7, 100), 7.0, dtype=torch.bfloat16, device=dev)
    mhc.mhc_mxfp4_restore(out, out=back[:6])
    assert (back[6] == 7).all()
    e = mhc.mhc_mxfp4(x[:0])
    assert e.codes.shape == (0, 64) and mhc.mhc_mxfp4_restore(e).shape == (0, 100)
