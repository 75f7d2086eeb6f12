"""Decode steps as a model runs them: block after block with fixed weights, each kernel started
while the one before it drains, eager and as a replayed graph; and an empty table."""
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
@pytest.mark.parametrize("M", [1, 5, 16])
def test_blocks_with_static_weights(M, bits):
    K, N, g, layers = 512, 1100, 64, 6
    gated, gemm = (w4.gated, w4.gemm) if bits == 4 else (w4.gated8, w4.gemm8)
    W = [(random_weights(N, K, g, bits, 3 * i), random_weights(N, K, g, bits, 3 * i + 1),
          random_weights(K, 1088, g, bits, 3 * i + 2)) for i in range(layers)]
    table = random_weights(300, K, g, bits, 99)
    embed = w4.embedding if bits == 4 else w4.embedding8
    ids = torch.zeros(M, dtype=torch.int64, device="cuda")

    def step(static):
        X = embed(ids, *table, g=g)
        for gate, up, down in W:
            H = gated(X, gate, up, g=g, act="gelu", static_weights=static)
            X = gemm(H[:, :1088].contiguous(), *down, g=g, static_weights=static)
            X = X / X.float().pow(2).mean().sqrt().bfloat16()
        return X

    seeds = range(4)
    want = []
    for s in seeds:
        ids.copy_(torch.randint(0, 300, (M,), generator=torch.Generator().manual_seed(s)))
        want.append(step(False))
        torch.cuda.synchronize()
    assert all(bool(x.isfinite().all()) for x in want) and not torch.equal(want[0], want[1])
    for s, x in zip(seeds, want):
        ids.copy_(torch.randint(0, 300, (M,), generator=torch.Generator().manual_seed(s)))
        for _ in range(5):
            assert torch.equal(step(True), x)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = step(True)
    for s, x in zip(seeds, want):
        ids.copy_(torch.randint(0, 300, (M,), generator=torch.Generator().manual_seed(s)))
        for _ in range(5):
            graph.replay()
        assert torch.equal(out, x)


def test_embedding_of_an_empty_table():
    none = tuple(t[:0].contiguous() for t in random_weights(4, 64, 64, 4, 1))
    ids = torch.tensor([-1, 0, 5], device="cuda")
    out = torch.full((3, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert bool((w4.embedding(ids, *none, g=64, out=out) == 0).all())
    assert w4.device_error() == 2
    assert w4.embedding_grad(out, ids, 0).shape == (0, 64)
    assert bool((w4.embedding(ids[:1], *none, g=64, out=out[:1]) == 0).all())     # padding alone is no error
