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
