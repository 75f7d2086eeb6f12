"""GPU parity of the gated feed-forward block, its backward pass and the linear layer's
gradients against plain products in binary64.

The weights are quantized and dequantized by the package itself (bit-exact with the host
oracle, tests/test_gpu_quantize.py and tests/test_gpu_w8a16.py), so every oracle here is a
binary64 product of the same bf16 values.  Bars: those of the GEMM (tests/helpers.py:
max 4e-3 of max|Y| against the unrounded result, Frobenius 1e-3 against the result
rounded to bf16), since each output is one rounding of a binary32 value.  dX is compared
with the product of the bf16 dG and dU, from which it is defined."""
import math

import numpy as np
import pytest
import torch

import workloads
import weight_only_quantization_rtn_b200 as w4
from weight_only_quantization_rtn_b200 import build as w4build
from helpers import assert_y_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    w4build.build()
    yield
    assert w4.device_error() == 0


def close(Y, Y64, what):
    assert Y.dtype == torch.bfloat16 and Y.shape == Y64.shape, what
    assert_y_close(workloads.bits(Y), Y64.cpu().numpy(), what)


def quantized(N, K, g, sym, bits, seed):
    """((codes, scales, zeros), dense weight in binary64)."""
    W = workloads.make_weight(N, K, 0.02, seed, outlier_frac=0.01, outlier_scale=20.0).cuda()
    q, dq = (w4.quantize, w4.dequantize) if bits == 4 else (w4.quantize8, w4.dequantize8)
    w = q(W, g, sym)
    return w, dq(*w, g=g, sym=sym).double()


def act64(x, kind):
    if kind == "silu":
        return x * torch.sigmoid(x)
    if kind == "gelu":
        return 0.5 * x * torch.erfc(-x / math.sqrt(2.0))
    if kind == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))
    return torch.relu(x)


def forward(bits):
    return w4.gated if bits == 4 else w4.gated8


def backward(bits):
    return w4.gated_backward if bits == 4 else w4.gated8_backward


def gated_case(M, N, K, g, sym, bits, act, seed, path="auto"):
    gg = g or K
    gate, Wg = quantized(N, K, gg, sym, bits, seed)
    up, Wu = quantized(N, K, gg, sym, bits, seed + 1)
    X = workloads.make_activation(M, K, seed + 2, outlier_frac=0.01, outlier_mode="scale",
                                  outlier_value=4.0).cuda()
    H, G, U = forward(bits)(X, gate, up, g=gg, sym=sym, act=act, save=True, path=path)
    G64, U64 = X.double() @ Wg.t(), X.double() @ Wu.t()
    what = f"M={M} N={N} K={K} g={g} sym={sym} bits={bits} {act} {path}"
    close(G, G64, "G " + what)
    close(U, U64, "U " + what)
    close(H, act64(G64, act) * U64, "H " + what)
    H2 = forward(bits)(X, gate, up, g=gg, sym=sym, act=act, path=path)
    assert torch.equal(H2, H), "without the projections: " + what
    return gate, up, Wg, Wu, X, H, G, U


SHAPES = [
    # one token to the decode kernel's most, odd feature counts, K of a few blocks
    (1, 11008, 4096, 128), (1, 1, 32, 32), (2, 7, 96, 32), (3, 130, 160, 0), (8, 1000, 1152, 128),
    (9, 257, 640, 64), (16, 515, 2304, 128), (5, 384, 11008, 0), (1, 8192, 256, 64),
    # tensor cores, one CTA per tile: every token tile and both sides of its border
    (17, 256, 256, 128), (31, 127, 96, 32), (32, 1000, 1184, 0), (33, 515, 1024, 64), (61, 2048, 4096, 64),
    (64, 129, 384, 128), (65, 640, 2048, 128), (100, 33, 32, 32), (128, 1, 512, 0),
    # pairs
    (129, 128, 256, 128), (200, 515, 1056, 0), (256, 257, 1024, 64), (257, 1111, 640, 32), (700, 300, 2112, 64),
]


@pytest.mark.parametrize("M,N,K,g", SHAPES)
@pytest.mark.parametrize("bits,sym,act", [(4, False, "silu"), (4, True, "gelu_tanh"), (8, False, "gelu"),
                                          (8, True, "relu")])
def test_gated(M, N, K, g, bits, sym, act):
    gated_case(M, N, K, g, sym, bits, act, seed=1000 + M + N + K)


@pytest.mark.parametrize("M,path", [(1, "tensorcore"), (16, "tensorcore"), (16, "decode")])
def test_gated_forced_path(M, path):
    gated_case(M, 640, 1024, 128, False, 4, "silu", seed=77, path=path)


def test_gated_large():
    gated_case(2048, 1500, 4096, 128, False, 4, "silu", seed=5)


@pytest.mark.parametrize("M,N,K,g", [(1, 256, 256, 128), (2, 7, 96, 32), (16, 515, 288, 0), (33, 1000, 512, 64),
                                     (64, 64, 1184, 0), (77, 130, 640, 128), (128, 257, 1024, 128), (130, 1, 32, 32),
                                     (200, 1111, 1056, 32), (333, 640, 2304, 64), (512, 2048, 4096, 128)])
@pytest.mark.parametrize("bits,sym,act", [(4, False, "silu"), (4, True, "gelu"), (8, False, "gelu_tanh"),
                                          (8, True, "relu")])
def test_gated_backward(M, N, K, g, bits, sym, act):
    gg = g or K
    seed = 2000 + M + N + K
    gate, Wg = quantized(N, K, gg, sym, bits, seed)
    up, Wu = quantized(N, K, gg, sym, bits, seed + 1)
    dH, G, U = (workloads.make_activation(M, N, seed + i).cuda() for i in (2, 3, 4))
    dX, dG, dU = backward(bits)(dH, G, U, gate, up, g=gg, sym=sym, act=act)
    G64 = G.double().requires_grad_(True)
    a64 = act64(G64, act)
    d64, = torch.autograd.grad(a64.sum(), G64)
    what = f"M={M} N={N} K={K} g={g} sym={sym} bits={bits} {act}"
    close(dG, dH.double() * U.double() * d64, "dG " + what)
    close(dU, dH.double() * a64.detach(), "dU " + what)
    close(dX, dG.double() @ Wg + dU.double() @ Wu, "dX " + what)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
def test_gate_gradient_against_differences(act):
    """dG and dU against central differences of act(g)·u.

    With a step h the difference of a function with |f'''| ≤ 4·|u| (these activations'
    third derivatives are below 4 at every point) is off by at most 4·|u|·h²/6 plus the
    binary64 cancellation, about 2^-52·|a·u|/h; the results are rounded to bf16 once
    (2^-8) from binary32 values that the approximate exponential leaves within 2^-18 of
    the terms they are summed from (at most 1.2·|u|)."""
    M, N, K = 64, 256, 64
    gate, _ = quantized(N, K, 64, False, 4, 1)
    up, _ = quantized(N, K, 64, False, 4, 2)
    G = torch.linspace(-9, 9, M * N, dtype=torch.float32).view(M, N).to(torch.bfloat16).cuda()
    if act == "relu":
        G = torch.where(G.abs() < 0.01, torch.full_like(G, 0.5), G)     # away from the kink
    U = workloads.make_activation(M, N, 3).cuda()
    dH = torch.ones_like(U)
    _, dG, dU = w4.gated_backward(dH, G, U, gate, up, g=64, act=act)
    g, u, h = G.double(), U.double(), 1e-4
    d = (act64(g + h, act) - act64(g - h, act)) / (2 * h) * u
    tol = d.abs() * 2.0 ** -8 + u.abs() * (1.2 * 2.0 ** -18 + 4 * h * h / 6 + 1e-10)
    assert bool(((dG.double() - d).abs() <= tol).all())
    a = act64(g, act)
    assert bool(((dU.double() - a).abs() <= a.abs() * 2.0 ** -8 + g.abs() * 2.0 ** -18).all())


@pytest.mark.parametrize("M,N,K,g", [(1, 512, 256, 128), (3, 9, 64, 32), (16, 1000, 11008, 0), (48, 77, 1184, 0),
                                     (64, 4096, 1152, 128), (77, 2048, 2048, 128), (128, 130, 320, 64),
                                     (129, 515, 1024, 32), (300, 1111, 640, 128), (520, 4096, 1024, 64)])
@pytest.mark.parametrize("bits,sym", [(4, False), (4, True), (8, False), (8, True)])
def test_gemm_dgrad(M, N, K, g, bits, sym):
    gg = g or K
    w, W = quantized(N, K, gg, sym, bits, 3000 + M)
    dY = workloads.make_activation(M, N, 3001 + N).cuda()
    f = w4.gemm_dgrad if bits == 4 else w4.gemm8_dgrad
    dX = f(dY, *w, g=gg, sym=sym)
    close(dX, dY.double() @ W, f"M={M} N={N} K={K} g={g} bits={bits} sym={sym}")
    assert torch.equal(dX, f(dY, *w, g=gg, sym=sym))


def test_gemm_dgrad_one_hot_reads_weights_exactly():
    """dY = identity rows returns Ŵ bit for bit, at every row and channel."""
    N, K, g = 320, 640, 128
    for bits, q, dq, f in ((4, w4.quantize, w4.dequantize, w4.gemm_dgrad),
                           (8, w4.quantize8, w4.dequantize8, w4.gemm8_dgrad)):
        w = q(workloads.make_weight(N, K, 0.02, 9).cuda(), g, False)
        eye = torch.eye(N, dtype=torch.bfloat16, device="cuda")
        assert torch.equal(f(eye, *w, g=g), dq(*w, g=g))


@pytest.mark.parametrize("M,N,K", [(1, 8, 32), (2, 1, 32), (5, 257, 96), (63, 130, 320), (64, 256, 256), (65, 300, 1184),
                                   (200, 1111, 640), (1000, 512, 2304), (2048, 777, 1024), (77, 4096, 4096)])
def test_gemm_wgrad(M, N, K):
    dY = workloads.make_activation(M, N, 41).cuda()
    X = workloads.make_activation(M, K, 42).cuda()
    dW = w4.gemm_wgrad(dY, X)
    close(dW, dY.double().t() @ X.double(), f"M={M} N={N} K={K}")
    assert torch.equal(dW, w4.gemm_wgrad(dY, X))


def test_empty_sizes():
    gate, _ = quantized(64, 128, 128, False, 4, 1)
    X = torch.zeros(0, 128, dtype=torch.bfloat16, device="cuda")
    assert w4.gated(X, gate, gate).shape == (0, 64)
    none = tuple(t[:0].contiguous() for t in gate)
    X = workloads.make_activation(3, 128, 1).cuda()
    assert w4.gated(X, none, none).shape == (3, 0)
    e = torch.empty(3, 0, dtype=torch.bfloat16, device="cuda")
    out = torch.full((3, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert bool((w4.gemm_dgrad(e, *none, out=out) == 0).all())
    out.fill_(float("nan"))
    dX, dG, dU = w4.gated_backward(e, e, e, none, none, out=out)
    assert bool((dX == 0).all()) and dG.shape == (3, 0) and dU.shape == (3, 0)
    out = torch.full((64, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    assert bool((w4.gemm_wgrad(e, torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"), out=out) == 0).all())


@pytest.mark.parametrize("M", [4, 40, 300])
def test_non_finite_activations_stay_in_their_row(M):
    """A NaN or infinity in one token reaches that token's outputs only."""
    N, K = 300, 256
    gate, Wg = quantized(N, K, 128, False, 4, 11)
    up, Wu = quantized(N, K, 128, False, 4, 12)
    X = workloads.make_activation(M, K, 13).cuda()
    clean = w4.gated(X, gate, up)
    X[1, 7], X[2, 250] = float("nan"), float("inf")
    H = w4.gated(X, gate, up)
    rows = torch.arange(M, device="cuda")
    keep = (rows != 1) & (rows != 2)
    assert torch.equal(H[keep], clean[keep])
    assert bool(H[1].isnan().all())
    dY = workloads.make_activation(M, N, 14).cuda()
    clean = w4.gemm_dgrad(dY, *gate)
    dY[1, 3] = float("nan")
    dX = w4.gemm_dgrad(dY, *gate)
    assert torch.equal(dX[rows != 1], clean[rows != 1]) and bool(dX[1].isnan().all())


def test_training_step_together():
    """Embedding, block, down projection, and the way back, as a training step runs them:
    every gradient against binary64 automatic differentiation of the same weights.

    The step's own intermediates are rounded to bf16 (2^-8 each), so the chain is compared
    with a bar that counts its roundings: E, H, dH, dG and dU, and the result itself, each
    at most 2^-8 of what it rounds; the sums they enter have norms that add at most
    linearly: six half steps of 2^-8."""
    V, K, N, T, g = 500, 256, 640, 300, 64
    table, Wt = quantized(V, K, g, False, 8, 21)
    gate, Wg = quantized(N, K, g, False, 4, 22)
    up, Wu = quantized(N, K, g, False, 4, 23)
    down, Wd = quantized(K, N, g, False, 4, 24)
    ids = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(3)).cuda()
    ids[-7:] = -1
    E = w4.embedding8(ids, *table, g=g, scale=8.0)
    H, G, U = w4.gated(E, gate, up, g=g, save=True)
    Y = w4.gemm(H, *down, g)
    dY = workloads.make_activation(T, K, 25).cuda()
    dH = w4.gemm_dgrad(dY, *down, g=g)
    dX, dG, dU = w4.gated_backward(dH, G, U, gate, up, g=g)
    grads = {"table": w4.embedding_grad(dX, ids, V, scale=8.0), "gate": w4.gemm_wgrad(dG, E),
             "up": w4.gemm_wgrad(dU, E), "down": w4.gemm_wgrad(dY, H)}
    p = {"table": Wt, "gate": Wg, "up": Wu, "down": Wd}
    p = {k: v.clone().requires_grad_(True) for k, v in p.items()}
    E64 = torch.where((ids >= 0)[:, None], p["table"][ids.clamp(min=0)] * 8.0, torch.zeros((), dtype=torch.float64,
                                                                                       device="cuda"))
    H64 = act64(E64 @ p["gate"].t(), "silu") * (E64 @ p["up"].t())
    Y64 = H64 @ p["down"].t()
    want = dict(zip(p, torch.autograd.grad((Y64 * dY.double()).sum(), list(p.values()))))
    for k, got in grads.items():
        off = (got.double() - want[k]).norm() / want[k].norm()
        assert off <= 6 * 2.0 ** -8, (k, float(off))
    off = (Y.double() - Y64.detach()).norm() / Y64.detach().norm()
    assert off <= 6 * 2.0 ** -8


def test_streams_and_graphs():
    """Two streams at once, and two captured graphs replayed at once, give what one call gives."""
    M, N, K = 40, 1000, 2048
    gate, _ = quantized(N, K, 128, False, 4, 31)
    up, _ = quantized(N, K, 128, False, 4, 32)
    Xs = [workloads.make_activation(m, K, 33 + i).cuda() for i, m in enumerate((M, 3))]
    dYs = [workloads.make_activation(m, N, 43 + i).cuda() for i, m in enumerate((M, 3))]
    want = [(w4.gated(X, gate, up), w4.gemm_dgrad(dY, *gate), w4.gemm_wgrad(dY, X)) for X, dY in zip(Xs, dYs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Xs]
    got = []
    for _ in range(3):
        for s, X, dY in zip(streams, Xs, dYs):
            with torch.cuda.stream(s):
                got.append((w4.gated(X, gate, up), w4.gemm_dgrad(dY, *gate), w4.gemm_wgrad(dY, X)))
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(r, want[i % 2]))
    graphs, outs = [], []
    for X, dY in zip(Xs, dYs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append((w4.gated(X, gate, up), w4.gemm_dgrad(dY, *gate), w4.gemm_wgrad(dY, X)))
        graphs.append(graph)
    for o in outs:
        for t in o:
            t.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(3):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for o, r in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, r))
