"""Rows so long that their byte offsets need more bits than their element indexes."""
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
    torch.cuda.empty_cache()


@pytest.mark.parametrize("K,dtype", [((1 << 29) + 64, torch.float32), ((1 << 30) + 64, torch.bfloat16)])
def test_embedding_grad(K, dtype):
    """Rows of 2 GB and more: those that no token names are zeros, the named one is its token's."""
    V = 5
    ids = torch.tensor([3], device="cuda")
    dY = torch.zeros(1, K, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1, 2**28 - 1, 2**28, K // 2, K - 1], device="cuda")
    dY[0, at] = torch.arange(1, 7, device="cuda").bfloat16()
    out = torch.full((V, K), float("nan"), dtype=dtype, device="cuda")
    w4.embedding_grad(dY, ids, V, dtype=dtype, out=out)
    for v in range(V):
        if v == 3:
            assert torch.equal(out[v], dY[0].to(dtype))
        else:
            assert int(out[v].count_nonzero()) == 0, v       # (a NaN is not zero)


def wide_weights(N, K, g, bits, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randint(0, 256, (N, K * bits // 8), generator=gen, dtype=torch.uint8, device="cuda"),
            (torch.rand(N, K // g, generator=gen, device="cuda") * 0.02 + 0.001).bfloat16(),
            torch.randint(0, 1 << bits, (N, K // g), generator=gen, device="cuda").bfloat16())


# codes that begin 2^31 bits into a row
WIDE = [(4, (1 << 29) + 4096), (8, (1 << 28) + 4096)]


@pytest.mark.parametrize("bits,K", WIDE)
def test_gated(bits, K):
    """One-hot tokens bring single weights out exactly."""
    M, N, g = 17, 2, 128
    gate, up = wide_weights(N, K, g, bits, 1), wide_weights(N, K, g, bits, 2)
    X = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    at = [0, 77, K // 2, K - 1] + [K - 1 - 257 * i for i in range(1, 14)]
    for m, k in enumerate(at):
        X[m, k] = 1.0
    f, dq = (w4.gated, w4.dequantize) if bits == 4 else (w4.gated8, w4.dequantize8)
    _, G, U = f(X, gate, up, g=g, save=True)
    del X
    for Y, w in ((G, gate), (U, up)):
        assert torch.equal(Y, dq(*w, g=g)[:, at].t())


@pytest.mark.parametrize("bits,K", WIDE)
def test_gemm_dgrad(bits, K):
    N, g = 3, 128
    w = wide_weights(N, K, g, bits, 3)
    f, dq = (w4.gemm_dgrad, w4.dequantize) if bits == 4 else (w4.gemm8_dgrad, w4.dequantize8)
    dX = f(torch.eye(N, dtype=torch.bfloat16, device="cuda")[:2].contiguous(), *w, g=g)
    W = dq(*w, g=g)
    assert all(torch.equal(dX[m], W[m]) for m in range(2))
