"""gemm_pair_kernel where a CTA goes through several tiles, or parts of tiles, whose numbers of
reduction blocks are no multiple of the dequantizing groups: the rings carry over from one to
the next.  Bars and oracle as in test_gpu_gated.py; every call is repeated and compared bit for bit."""
import pytest
import torch

import workloads
import weight_only_quantization_rtn_b200 as w4
from weight_only_quantization_rtn_b200 import build as w4build
from test_gpu_gated import act64, close, forward
from test_gpu_train_paths import random_weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    w4build.build()
    yield
    assert w4.device_error() == 0


def gated_repeated(M, N, K, g, bits, path="auto", times=6):
    g = g or K
    gate, up = random_weights(N, K, g, bits, M + K), random_weights(N, K, g, bits, M + K + 1)
    dq = w4.dequantize if bits == 4 else w4.dequantize8
    X = workloads.make_activation(M, K, 3).cuda()
    H, G, U = forward(bits)(X, gate, up, g=g, save=True, path=path)
    G64, U64 = X.double() @ dq(*gate, g=g).double().t(), X.double() @ dq(*up, g=g).double().t()
    what = f"M={M} N={N} K={K} g={g} bits={bits}"
    close(G, G64, "G " + what)
    close(U, U64, "U " + what)
    close(H, act64(G64, "silu") * U64, "H " + what)
    for _ in range(times):
        again = forward(bits)(X, gate, up, g=g, save=True, path=path)
        assert all(torch.equal(a, b) for a, b in zip(again, (H, G, U))), what


# whole tiles, one to three per CTA: 5, 6, 7, 19 and 10 blocks of 64
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M", [61, 65, 80, 96])
@pytest.mark.parametrize("K,g", [(320, 64), (384, 128), (448, 64), (1184, 32), (640, 0)])
@pytest.mark.parametrize("N", [19200, 40000])
def test_whole_tiles(M, N, K, g, bits):
    gated_repeated(M, N, K, g, bits)


# tiles of one, two and three blocks
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M,path", [(3, "tensorcore"), (16, "tensorcore"), (20, "auto"), (40, "auto"), (64, "auto"), (90, "auto")])
@pytest.mark.parametrize("K", [32, 64, 96, 160])
def test_short_tiles(M, path, K, bits):
    gated_repeated(M, 60000, K, 32, bits, path)


# tiles shared by CTAs whose shares do not begin with a tile
@pytest.mark.parametrize("bits,M,N,K", [(8, 80, 11008, 4096), (4, 80, 11008, 4096), (8, 61, 11008, 4096), (8, 96, 4096, 8192),
                                        (4, 96, 11008, 4160), (4, 61, 5000, 4032)])
def test_shared_tiles(bits, M, N, K):
    gated_repeated(M, N, K, 64, bits)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M", [20, 77, 96])
@pytest.mark.parametrize("N", [300, 512, 640, 64])
def test_gradient_tiles(M, N, bits):
    """dX of several tiles per CTA, 1 to 10 blocks each."""
    K, g = 81920, 128
    w = random_weights(N, K, g, bits, N)
    dq, f = (w4.dequantize, w4.gemm_dgrad) if bits == 4 else (w4.dequantize8, w4.gemm8_dgrad)
    dY = workloads.make_activation(M, N, 5).cuda()
    dX = f(dY, *w, g=g)
    close(dX, dY.double() @ dq(*w, g=g).double(), f"M={M} N={N} bits={bits}")
    for _ in range(6):
        assert torch.equal(f(dY, *w, g=g), dX)
