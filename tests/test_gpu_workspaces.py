"""Workspaces that hold what earlier calls may have left there: anything at all, ready flags of
other launches included."""
import pytest
import torch

import workloads
import weight_only_quantization_rtn_b200 as w4
from weight_only_quantization_rtn_b200 import build as w4build
from test_gpu_train_paths import random_weights

pytestmark = pytest.mark.gpu

# 64-bit words: nothing, all ones, and the values that marked a part ready in every launch
WORDS = [0, -1, 0x9E6C63D07F8A5C3D - (1 << 64), 0x7F8A5C3D7F8A5C3D]


@pytest.fixture(scope="module", autouse=True)
def _built():
    w4build.build()
    yield
    assert w4.device_error() == 0


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("M", [20, 77, 200])
@pytest.mark.parametrize("word", WORDS)
def test_shared_tiles_of_the_gradient(M, word):
    N, K, g = 4096, 512, 128
    w = random_weights(N, K, g, 4, 3)
    dY = workloads.make_activation(M, N, 4).cuda()
    want = w4.gemm_dgrad(dY, *w, g=g)
    L = w4.lib()
    nbytes = L.w4a16_gemm_dgrad_workspace_size(M, N, K, g)
    assert nbytes > 0                                         # tiles are shared
    ws = torch.full((nbytes // 8,), word, dtype=torch.int64, device="cuda")
    dX = torch.empty_like(want)
    for _ in range(3):
        assert L.w4a16_gemm_dgrad(dY.data_ptr(), M, N, *(t.data_ptr() for t in w), K, g, 0, dX.data_ptr(), ws.data_ptr(),
                                  nbytes, stream()) == 0
        assert torch.equal(dX, want)
        ws.fill_(word)


@pytest.mark.parametrize("bits,M", [(4, 1), (4, 8), (4, 16), (8, 5)])
@pytest.mark.parametrize("word", WORDS)
def test_shared_row_blocks_of_the_gated_block(M, bits, word):
    N, K, g = 1000, 4096, 128
    gate, up = random_weights(N, K, g, bits, 3), random_weights(N, K, g, bits, 4)
    X = workloads.make_activation(M, K, 5).cuda()
    f = w4.gated if bits == 4 else w4.gated8
    want = f(X, gate, up, g=g, path="decode")
    L = w4.lib()
    size, call = ((L.w4a16_gated_workspace_size, L.w4a16_gated) if bits == 4 else
                  (L.w8a16_gated_workspace_size, L.w8a16_gated))
    nbytes = size(M, N, K, g, w4.PATH_DECODE)
    assert nbytes > 0
    ws = torch.full((nbytes // 8,), word, dtype=torch.int64, device="cuda")
    H = torch.empty_like(want)
    for _ in range(3):
        assert call(X.data_ptr(), M, K, *(t.data_ptr() for t in gate), *(t.data_ptr() for t in up), N, g, 0, 0,
                    H.data_ptr(), None, None, ws.data_ptr(), nbytes, w4.PATH_DECODE, stream()) == 0
        assert torch.equal(H, want)
        ws.fill_(word)


@pytest.mark.parametrize("M,N", [(1500, 2048), (1500, 2047)])
@pytest.mark.parametrize("swap", [False, True])
def test_gate_gradient_over_its_inputs(M, N, swap):
    """dG and dU in G's and U's memory (or the other way round), each thread going through many
    elements, several calls in a row."""
    K, g = 64, 32
    w = random_weights(N, K, g, 4, 6)
    dH, G0, U0 = (workloads.make_activation(M, N, s).cuda() for s in (1, 2, 3))
    want = w4.gated_backward(dH, G0, U0, w, w, g=g)
    L = w4.lib()
    nbytes = L.w4a16_gated_backward_workspace_size(M, N, K, g)
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")
    ptrs = [t.data_ptr() for t in w]
    for _ in range(4):
        G, U = G0.clone(), U0.clone()
        dG, dU = (U, G) if swap else (G, U)
        dX = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
        assert L.w4a16_gated_backward(dH.data_ptr(), G.data_ptr(), U.data_ptr(), M, N, *ptrs, *ptrs, K, g, 0, 0,
                                      dX.data_ptr(), dG.data_ptr(), dU.data_ptr(), ws.data_ptr(), nbytes, stream()) == 0
        assert all(torch.equal(a, b) for a, b in zip(want, (dX, dG, dU)))
