"""The products with 4-bit weights in tiles on the GPU, at sizes for which the launch plan takes them (tests/test_experts_tiles_host.py),
against the definition in 64 bits; the errors are those of tests/test_gpu_experts.py."""
import sys

import numpy as np
import pytest

from experts_helpers import U, check, mxfp4, to_mxfp4, values
from experts_tiles import DOWN
from gpu_helpers import device
from test_gpu_experts import a_plan, part_error, some_experts, to_dev

pytestmark = pytest.mark.gpu


def case(text):
    print(f"[case] {text}", file=sys.stderr, flush=True)


def pairs_of(x, w, flat, tok):
    """x[tok[p]] w[flat[p]]^T for each pair p with an expert, zeros for the others."""
    out = np.zeros((len(flat), w.shape[1]))
    for e in np.unique(flat[flat >= 0]):
        at = flat == e
        out[at] = x[tok[at]] @ w[e].T
    return out


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("T,k,E,D,F,shape", DOWN)
def test_finite_results_beside_a_nan_or_an_infinity(T, k, E, D, F, shape, f16):
    # A weight row with a block of NaN spoils its column of y for its expert's tokens, and one whose sums overflow makes them
    # infinite; the columns beside them are those of weights without either. Whole numbers, whose fp32 sums are exact.
    import mhc_hyper_connection_amd as mhc
    import torch
    dev = device()
    rng = np.random.default_rng(T + D)
    case(f"finite beside NaN T={T} k={k} E={E} D={D} F={F} f16={f16}")
    e = some_experts(rng, T, k, E, masked=True)
    flat = e.reshape(-1)
    h, w = mxfp4(rng, T, k, F, low=127, high=129), mxfp4(rng, E, D, F, low=127, high=129)
    h[0][..., 0] = h[0][..., 0] & 0xF0 | 7                   # 6 at the first place
    nan, inf = [37, D - 3], [44, D - 7]                      # two in one run of 32 each; the last run is short
    w[0][0, nan] = w[0][1, inf] = 0
    wt = (1 + rng.integers(0, 4, (T, k))).astype(np.float32) / 4
    p, hm, wd = a_plan(e, E, dev), to_mxfp4(*h, F, f16, dev), to_dev(wt, dev)
    clean = mhc.mhc_experts_down(hm, p, wd, to_mxfp4(*w, F, f16, dev))
    hv, wv = values(*h, F).reshape(T * k, F), values(*w, F)
    y = pairs_of(hv, wv, flat, np.arange(T * k))
    err = np.zeros_like(y) if f16 else part_error(y)
    weighted = lambda v: (wt.astype(float).reshape(T * k, 1) * v).reshape(T, k, D).sum(1)
    check("clean", clean, weighted(y), weighted(err) + (k + 1) * U * weighted(np.abs(y)), f16)

    w[1][0, nan, 1] = 255                                    # a block of the reduction's second 32 values
    w[0][1, inf, 0], w[1][1, inf, 0] = 7, 254                # 6 2^127 6 2^0, or 2^1, is past fp32's range
    got = mhc.mhc_experts_down(hm, p, wd, to_mxfp4(*w, F, f16, dev)).cpu()
    clean = clean.cpu()
    has = lambda x: torch.from_numpy((e == x).any(1))
    rest = torch.ones(D, dtype=torch.bool)
    rest[nan + inf] = False
    assert has(0).any() and has(1).any() and (~has(0)).any() and (~has(1)).any()
    assert torch.equal(got[:, rest], clean[:, rest])
    assert torch.isnan(got[:, nan][has(0)]).all() and torch.equal(got[:, nan][~has(0)], clean[:, nan][~has(0)])
    assert (got[:, inf][has(1)] == float("inf")).all() and torch.equal(got[:, inf][~has(1)], clean[:, inf][~has(1)])
