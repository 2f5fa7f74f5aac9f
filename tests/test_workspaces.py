"""The workspaces of calls that may run at the same time, on the host: the library call is replaced by one that notes its
arguments, so nothing is launched."""
import contextlib

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


@pytest.mark.parametrize("checkpoint", [False, True])
def test_backward_runs_with_its_tensors_device_current(monkeypatch, checkpoint):
    # as on a second GPU while the first is the current one
    current = []

    @contextlib.contextmanager
    def on_gpu(device):
        current.append(device)
        yield
        current.pop()

    def launch(*args):
        assert current == [torch.device("cpu")]      # the tensors' device here
        return mhc.MHC_OK

    monkeypatch.setattr(mhc, "raw_backward", launch)
    monkeypatch.setattr(mhc, "raw_backward_checkpoint", launch)
    monkeypatch.setattr(mhc, "_stream", lambda device: None)
    monkeypatch.setattr(mhc, "_on_gpu", on_gpu)
    mhc.mhc_pre_backward(*backward_inputs(checkpoint))


@pytest.fixture
def forward(monkeypatch):
    """mhc_pre on tensors of a size, on a stream of that handle or in a capture of that number: the workspace it took."""
    where = {"stream": 0, "capture": 0}
    seen = []

    class Device:           # a GPU's name over host memory
        type, index = "cuda", 0

    gpu = Device()

    def make(*a, device, **k):
        return real(*a, device="cpu", **k)

    def launch(params, ptrs, ws, ws_bytes, stream):
        seen.append((ws, ws_bytes))
        return mhc.MHC_OK

    real = mhc.PreForward
    monkeypatch.setattr(mhc, "PreForward", make)
    monkeypatch.setattr(mhc, "raw_forward", launch)
    monkeypatch.setattr(mhc, "_raw_stream", lambda device: where["stream"])
    monkeypatch.setattr(mhc, "_capturing", lambda device: where["capture"] != 0)
    monkeypatch.setattr(mhc, "capture_id", lambda stream: where["capture"] if where["capture"] > 0 else 0)
    monkeypatch.setattr(mhc, "_RUNNERS", {})
    monkeypatch.setattr(mhc, "_GRAPH_RUNNERS", {})
    keep = []

    def call(tokens, stream, capture=0):
        where.update(stream=stream, capture=capture)
        r = mhc._runner(tokens, N, D, 3, 20, 1e-6, 1e-6, False, gpu)
        keep.append(r)
        z = torch.zeros
        r(z((tokens, N, D), dtype=torch.bfloat16), z((M, N * D)), z(3), z(M))
        return seen[-1]

    return call


def test_forward_calls_on_different_streams_share_no_workspace(forward):
    first, second, default = forward(T, 16), forward(T, 32), forward(T, 0)
    assert len({first, second, default}) == 3
    assert forward(T, 16) == first and forward(T, 32) == second and forward(T, 0) == default


def test_graphs_share_no_workspace_with_eager_calls_or_each_other(forward):
    eager, other = forward(T, 16), forward(T, 32)
    a = forward(T, 48, capture=1)
    assert a == other and forward(T, 48, capture=1) == a      # the last eager call's, zero-filled and used before; the same all through the graph
    b = forward(T, 48, capture=2)
    assert b == eager
    c, d = forward(T, 48, capture=3), forward(T, 48, capture=3)
    again, more = forward(T, 16), forward(T, 32)              # eager calls have new ones
    assert len({a, b, c, d, again, more}) == 6
    assert forward(T, 48, capture=1) == a and forward(T, 16) == again
    e = forward(T + 1, 16)
    assert forward(T, 48, capture=4) in (again, more) and forward(T + 1, 16) == e      # of its own size


def test_a_capture_without_a_number_takes_no_eager_workspace(forward):
    eager = forward(T, 16)
    a, b = forward(T, 48, capture=-1), forward(T, 48, capture=-1)
    assert len({eager, a, b}) == 3 and forward(T, 16) == eager


def test_forward_keeps_few_launchers(forward):
    for tokens in range(1, 2 * mhc._MAX_RUNNERS):
        forward(tokens, 0)
    assert len(mhc._RUNNERS) <= mhc._MAX_RUNNERS
    for capture in range(1, 2 * mhc._MAX_RUNNERS):
        forward(T, 0)
        forward(T, 48, capture=capture)
    assert len(mhc._GRAPH_RUNNERS) <= mhc._MAX_RUNNERS
