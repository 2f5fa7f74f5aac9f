"""Calls of one size that run at the same time, on the GPU: the pre-mapping's backward from 16-bit x on several streams, and
captured into two graphs that are replayed on streams of their own beside eager calls. Every result equals the call's own
when it runs alone, bit for bit."""
import sys

import pytest

from gpu_helpers import device
from test_gpu_sublayer import SubLayer

pytestmark = pytest.mark.gpu


def bits(out):
    import torch
    return {k: v.clone().view(torch.uint8) for k, v in out.items()}


def same(out, want):
    import torch
    return all(torch.equal(out[k].view(torch.uint8), want[k]) for k in want)


def pre_backward(L, p):
    import mhc_hyper_connection_amd as mhc
    s = L.saved
    return mhc.mhc_pre_backward(L.x, L.phi, L.alpha, p["grad_x"], p["grad_post"], p["grad_comb"], s["inv_rms"], s["h_mix"], s["h_pre"], L.h_post,
                                L.gamma, p["grad_residual"], num_iters=L.iters, sum_out=s["sum_out"], norm_out=s["norm_out"])


def layers_and_gradients(seeds):
    import mhc_hyper_connection_amd as mhc
    layers = [SubLayer(1400, 4, 264, 64, False, seed=s, iters=2) for s in seeds]
    grads, want = [], []
    for L in layers:
        L.forward()
        grads.append(mhc.mhc_post_backward(L.grad_out, L.y, L.x, L.h_post, L.h_res))
        want.append(bits(pre_backward(L, grads[-1])))
    return layers, grads, want


def test_streams():
    import torch
    print("[case] 16-bit backward on streams", file=sys.stderr, flush=True)
    layers, grads, want = layers_and_gradients((1, 2, 3))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(device()) for _ in layers]
    for _ in range(3):
        got = []
        for L, g, s in zip(layers, grads, streams):
            with torch.cuda.stream(s):
                got.append(pre_backward(L, g))
        torch.cuda.synchronize()
        assert all(same(g, w) for g, w in zip(got, want))


def test_graphs_beside_eager_calls():
    import torch
    print("[case] 16-bit backward in graphs", file=sys.stderr, flush=True)
    layers, grads, want = layers_and_gradients((4, 5, 6))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for L, g in zip(layers[:2], grads):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(pre_backward(L, g))
        graphs.append(graph)
    streams = [torch.cuda.Stream(device()) for _ in range(3)]
    for rep in range(4):
        for o in outs:
            for v in o.values():
                v.view(torch.uint8).fill_(0x7F)
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        with torch.cuda.stream(streams[2]):
            eager = pre_backward(layers[2], grads[2])
        torch.cuda.synchronize()
        assert all(same(o, w) for o, w in zip((*outs, eager), want)), rep


def forward_inputs(T, D, seed):
    import synth
    from gpu_helpers import to_dev
    inp = synth.custom(T, 4, D, need_backward=True, seed=seed)
    return [to_dev(a, device()) for a in (inp.x, inp.phi, inp.alpha, inp.bias)]


def forward(args):
    import mhc_hyper_connection_amd as mhc
    h_in, h_post, h_res, extras = mhc.mhc_pre(*args, need_backward=True)
    return {"h_in": h_in, "h_post": h_post, "h_res": h_res, **extras}


@pytest.mark.parametrize("T,D", [(1400, 264), (4096, 1024)])
def test_forward_on_streams(T, D):
    # sizes of the classic and the streaming path: workgroups that do not wait on each other
    import torch
    print(f"[case] forward on streams T={T} D={D}", file=sys.stderr, flush=True)
    args = [forward_inputs(T, D, seed) for seed in (1, 2, 3)]
    want = [bits(forward(a)) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(device()) for _ in args]
    for _ in range(3):
        got = []
        for a, s in zip(args, streams):
            with torch.cuda.stream(s):
                got.append(forward(a))
        torch.cuda.synchronize()
        assert all(same(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("T,D", [(60, 1056), (1300, 264), (4100, 1024)])
def test_forward_first_called_under_capture(T, D):
    # of sizes that no call had before: the captured calls' workspaces serve them alone
    import torch
    print(f"[case] forward under capture T={T} D={D}", file=sys.stderr, flush=True)
    args = [forward_inputs(T, D, seed) for seed in (1, 2)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for a in args:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(forward(a))
        graphs.append(graph)
    torch.cuda.synchronize()
    want = [bits(forward(a)) for a in args]
    for rep in range(4):
        for o in outs:
            for v in o.values():
                v.view(torch.uint8).fill_(0x7F)
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
        eager = [forward(a) for a in args]
        torch.cuda.synchronize()
        assert all(same(o, w) for o, w in zip(outs + eager, want + want)), rep


@pytest.mark.parametrize("T,D", [(60, 1088), (1300, 264), (4100, 1024)])
def test_forward_captured_after_eager_calls(T, D):
    # the first graph takes the eager calls' workspace, the second has one of its own, later eager calls have a new one: replayed
    # at the same time on streams of their own where no workgroups wait on each other (T > 64)
    import torch
    print(f"[case] forward captured after eager calls T={T} D={D}", file=sys.stderr, flush=True)
    args = [forward_inputs(T, D, seed) for seed in (1, 2, 3)]
    want = [bits(forward(a)) for a in args]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for a in args[:2]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            first = forward(a)
            outs.append({**{"2 " + k: v for k, v in forward(a).items()}, **first})      # two calls in one graph
        graphs.append(graph)
    want2 = [{**{"2 " + k: v for k, v in w.items()}, **w} for w in want[:2]]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(device()) for _ in range(3)]
    for rep in range(4):
        for o in outs:
            for v in o.values():
                v.view(torch.uint8).fill_(0x7F)
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
            if T <= 64:
                torch.cuda.synchronize()
        with torch.cuda.stream(streams[2]):
            eager = forward(args[2])
        torch.cuda.synchronize()
        assert same(eager, want[2]) and all(same(o, w) for o, w in zip(outs, want2)), rep


def test_captures_are_told_apart():
    import torch
    from mhc_hyper_connection_amd import _binding as B
    dev = device()
    numbers = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            numbers.append([B.capture_id(torch.cuda.current_stream(dev).cuda_stream) for _ in range(2)])
            torch.zeros(8, device=dev)
    assert numbers[0][0] == numbers[0][1] > 0 and numbers[1][0] == numbers[1][1] > 0 and numbers[0][0] != numbers[1][0]
    assert B.capture_id(torch.cuda.current_stream(dev).cuda_stream) == 0
