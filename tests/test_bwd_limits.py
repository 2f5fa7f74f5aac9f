"""The most tokens that the pre-mapping's backward takes, on the host: a size is either launchable or refused, by the
workspace query and by both calls."""
import pytest

from mhc_hyper_connection_amd import _binding as B

FAKE = 0x10000   # never dereferenced: every call here is refused
MOST = 4 * 0xFFFFFF   # one wave of 64 threads a token, at most 2^32 - 1 threads a grid


@pytest.mark.parametrize("n,num_iters", [(4, 0), (6, 3), (8, 20)])
def test_more_tokens_than_a_grid_holds_are_refused(n, num_iters):
    assert B.bwd_workspace_size(B.make_bwd_params(MOST, n, 8, num_iters=num_iters)) > MOST
    p = B.make_bwd_params(MOST + 1, n, 8, num_iters=num_iters)
    with pytest.raises(B.MhcError) as err:
        B.bwd_workspace_size(p)
    assert err.value.status == B.MHC_ERR_PARAM_INVALID
    ptrs = {f: FAKE for f in B.BWD_TENSOR_FIELDS}
    # the workspace is one byte short as well, so that no launch could follow
    assert B.raw_backward(p, ptrs, FAKE, 1, None) == B.MHC_ERR_PARAM_INVALID
    assert B.raw_backward_checkpoint(p, {**ptrs, "x": None}, FAKE, FAKE, FAKE, 1, None) == B.MHC_ERR_PARAM_INVALID
