"""GPU parity of the quantized embedding and its table's gradient.

A lookup is bit-exact: the row that dequantize gives, times the scale, rounded once.  The
gradient is compared with binary64 sums: n binary32 additions are off by at most
n·2^-24·Σ|dY|, the product with the scale by 2^-24, and a bf16 result by 2^-8 more."""
import pytest
import torch

import workloads
import weight_only_quantization_rtn_b200 as w4
from weight_only_quantization_rtn_b200 import build as w4build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    w4build.build()
    yield
    assert w4.device_error() == 0


def ids_of(T, V, kind, seed=0):
    gen = torch.Generator().manual_seed(seed)
    if kind == "same":
        ids = torch.full((T,), V // 2)
    elif kind == "tail":
        ids = (float(V) ** torch.rand(T, generator=gen, dtype=torch.float64) - 1).long().clamp(0, V - 1)
    else:
        ids = torch.randint(0, V, (T,), generator=gen)
    if kind == "pad":
        ids[torch.rand(T, generator=gen) < 0.4] = -1
    if kind == "allpad":
        ids[:] = -3
    return ids.cuda()


@pytest.mark.parametrize("T,V,K,g", [(1, 1, 32, 32), (16, 1000, 4096, 128), (7, 33, 160, 0), (300, 500, 1152, 64),
                                     (2, 40, 11008, 128), (1000, 257, 96, 32)])
@pytest.mark.parametrize("bits,sym", [(4, False), (4, True), (8, False), (8, True)])
@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_embedding_is_exact(T, V, K, g, bits, sym, scale):
    gg = g or K
    q, dq, f = ((w4.quantize, w4.dequantize, w4.embedding) if bits == 4 else
                (w4.quantize8, w4.dequantize8, w4.embedding8))
    w = q(workloads.make_weight(V, K, 0.02, V + K).cuda(), gg, sym)
    W = dq(*w, g=gg, sym=sym)
    for dt in (torch.int64, torch.int32):
        ids = ids_of(T, V, "pad", T).to(dt)
        want = (W[ids.clamp(min=0).long()].float() * scale).to(torch.bfloat16)
        want[ids < 0] = 0
        assert torch.equal(f(ids, *w, g=gg, sym=sym, scale=scale), want)
    if T % 2 == 0:
        assert torch.equal(f(ids.view(2, T // 2), *w, g=gg, sym=sym, scale=scale), want.view(2, T // 2, K))


def test_bad_ids_are_zeros_and_reported():
    w = w4.quantize(workloads.make_weight(10, 64, 0.02, 1).cuda(), 64, False)
    ids = torch.tensor([3, 10, 1 << 40, -1, 9], device="cuda")
    assert w4.device_error() == 0
    E = w4.embedding(ids, *w, g=64)
    assert w4.device_error() == 2 and w4.device_error() == 0
    W = w4.dequantize(*w, g=64)
    assert bool((E[1:4] == 0).all()) and torch.equal(E[0], W[3]) and torch.equal(E[4], W[9])
    dY = torch.ones(5, 64, dtype=torch.bfloat16, device="cuda")
    dW = w4.embedding_grad(dY, ids, 10)
    assert w4.device_error() == 2
    want = torch.zeros(10, 64, device="cuda")
    want[3] = want[9] = 1
    assert torch.equal(dW, want)


@pytest.mark.parametrize("T,V,K", [(1, 1, 32), (1, 1000, 32), (31, 5, 64), (32, 40, 96), (33, 2, 1024), (500, 32, 1056),
                                   (4096, 300, 256), (4097, 1, 64), (5000, 70000, 32), (9000, 4, 2080),
                                   (20000, 1000, 128)])
@pytest.mark.parametrize("kind", ["uniform", "tail", "same", "pad", "allpad"])
@pytest.mark.parametrize("dtype,scale", [(torch.float32, 1.0), (torch.bfloat16, 3.0)])
def test_embedding_grad(T, V, K, kind, dtype, scale):
    ids = ids_of(T, V, kind, T + V)
    dY = workloads.make_activation(T, K, 7).cuda()
    out = torch.full((V, K), float("nan"), dtype=dtype, device="cuda")
    dW = w4.embedding_grad(dY, ids, V, scale=scale, dtype=dtype, out=out)
    keep = ids >= 0
    want = torch.zeros(V, K, dtype=torch.float64, device="cuda")
    mag = torch.zeros(V, K, dtype=torch.float64, device="cuda")
    want.index_add_(0, ids[keep], dY[keep].double())
    mag.index_add_(0, ids[keep], dY[keep].double().abs())
    n = torch.zeros(V, dtype=torch.float64, device="cuda").index_add_(0, ids[keep], torch.ones_like(ids[keep]).double())
    tol = mag * (n[:, None] + 1) * 2.0 ** -24 * scale
    want = want * scale
    tol = tol + want.abs() * (2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8)
    assert bool(((dW.double() - want).abs() <= tol).all())
    assert torch.equal(w4.embedding_grad(dY, ids.int(), V, scale=scale, dtype=dtype), dW)


def test_embedding_grad_shapes_and_streams():
    ids = ids_of(600, 100, "tail").view(3, 200)
    dY = workloads.make_activation(600, 64, 5).cuda().view(3, 200, 64)
    want = w4.embedding_grad(dY, ids, 100)
    torch.cuda.synchronize()
    outs = []
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            outs.append(w4.embedding_grad(dY, ids, 100))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured = w4.embedding_grad(dY, ids, 100)
    captured.fill_(float("nan"))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs + [captured])
    empty = torch.empty(0, dtype=torch.int64, device="cuda")
    out = torch.full((10, 64), float("nan"), device="cuda")
    assert bool((w4.embedding_grad(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), empty, 10, out=out) == 0).all())
