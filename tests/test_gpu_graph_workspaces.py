"""Linear-layer calls captured into two graphs on one stream have workspaces of their own: the
graphs replayed at once on two streams give what single calls give."""
import pytest
import torch

import workloads
import weight_only_quantization_rtn_b200 as w4
from weight_only_quantization_rtn_b200 import build as w4build
from test_gpu_train_paths import random_weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    w4build.build()
    yield
    assert w4.device_error() == 0


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M", [1, 8, 40])
def test_two_graphs_at_once(M, bits):
    N, K, g = 1000, 8192, 128
    w = random_weights(N, K, g, bits, 1)
    gemm = w4.gemm if bits == 4 else w4.gemm8
    Xs = [workloads.make_activation(M, K, 2 + i).cuda() for i in range(2)]
    want = [gemm(X, *w, g=g) for X in Xs]
    graphs = []
    torch.cuda.synchronize()
    for X in Xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = [gemm(X, *w, g=g) for _ in range(4)]
        graphs.append((graph, outs))
    streams = [torch.cuda.Stream() for _ in Xs]
    for _ in range(20):
        for s, (graph, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (_, outs), y in zip(graphs, want):
        assert all(torch.equal(o, y) for o in outs)
    assert torch.equal(gemm(Xs[0], *w, g=g), want[0])


def test_captured_workspaces_are_not_kept():
    """A workspace that a capture allocated belongs to its graph, so no later call is given it."""
    N, K, g = 1000, 8192, 128
    w = random_weights(N, K, g, 4, 1)
    X = workloads.make_activation(3, K, 2).cuda()
    want = w4.gemm(X, *w, g=g)
    kept = {k: t.data_ptr() for k, t in w4._workspaces.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = w4.gemm(X, *w, g=g)
    assert {k: t.data_ptr() for k, t in w4._workspaces.items()} == kept
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_host_operands_captured():
    """Host to host in two graphs replayed at once: each has its own device buffers."""
    N, K, g, M = 1000, 4096, 128, 2
    w = random_weights(N, K, g, 4, 1)
    Xs = [workloads.make_activation(M, K, 5 + i).pin_memory() for i in range(2)]
    Ys = [torch.empty(M, N, dtype=torch.bfloat16, pin_memory=True) for _ in range(2)]
    want = [w4.gemm(X, *w, g=g).clone() for X in Xs]
    torch.cuda.synchronize()
    graphs = []
    for X, Y in zip(Xs, Ys):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            w4.gemm(X, *w, g=g, out=Y, sync=False)
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in Xs]
    for _ in range(20):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(Y, y) for Y, y in zip(Ys, want))
