"""The workspaces of calls that may run at the same time, on the host: the library call is replaced by one that notes its
arguments, so nothing is launched."""
import pytest

torch = pytest.importorskip("torch")
import mhc_hyper_connection_amd as mhc

T, N, D = 5, 4, 64
M = N * N + 2 * N


def backward_inputs(checkpoint):
    z = torch.zeros
    bf = torch.bfloat16
    x = z((T, N, D), dtype=bf)
    if checkpoint:
        x = mhc.Checkpoint(z((T, N, D), dtype=torch.int8), z((T, N, D // 32), dtype=torch.uint8), bf)
    return (x, z((M, N * D)), z(3), z((T, D), dtype=bf), z((T, N)), z((T, N, N)), z(T), z((T, M)), z((T, N)), z((T, N)))


@pytest.mark.parametrize("checkpoint", [False, True])
def test_backward_calls_in_flight_share_no_workspace(monkeypatch, checkpoint):
    # a second call of the same size is made while the first is under way, as on another stream
    seen = []

    def launch(params, ptrs, *rest):
        ws, size = rest[-3], rest[-2]
        seen.append((ws, size))
        if len(seen) < 3:
            mhc.mhc_pre_backward(*backward_inputs(checkpoint))
        return mhc.MHC_OK

    import contextlib
    monkeypatch.setattr(mhc, "raw_backward", launch)
    monkeypatch.setattr(mhc, "raw_backward_checkpoint", launch)
    monkeypatch.setattr(mhc, "_stream", lambda device: None)
    monkeypatch.setattr(mhc, "_on_gpu", lambda device: contextlib.nullcontext())
    mhc.mhc_pre_backward(*backward_inputs(checkpoint))
    assert len(seen) == 3
    for i, (a, size) in enumerate(seen):
        assert size > 0 and a % 64 == 0
        for b, other in seen[:i]:
            assert a + size <= b or b + other <= a, "two calls in flight write to one workspace"
