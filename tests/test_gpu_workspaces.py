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
