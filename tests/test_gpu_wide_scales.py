"""Scales over the whole bf16 range in the decode kernel: one-hot tokens bring Ŵ out bit for bit
(every other term is 0 times a finite weight), as dequantize gives it, for scales far below 1
and up to 2^127, beside rows of ordinary ones."""
import pytest
import torch

import weight_only_quantization_rtn_b200 as w4
from weight_only_quantization_rtn_b200 import build as w4build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    w4build.build()
    yield
    assert w4.device_error() == 0


def weights(N, K, g, bits, sym, exponent, seed):
    """Rows 0 .. N/2 with scales in [2^exponent, 2^(exponent + 1)), the others about 2^-8; codes
    around the zero point, so far off that every weight is finite."""
    gen = torch.Generator().manual_seed(seed)
    groups = K // g
    s = torch.ldexp(1 + torch.rand(N, groups, generator=gen), torch.tensor(exponent)).bfloat16()
    s = torch.where(s < 2.0 ** exponent * 1.99, s, torch.full_like(s, 2.0 ** exponent))
    s[N // 2:] = 2.0 ** -8
    far = max(1, min(1 << (bits - 1), 1 << max(0, 126 - exponent)) - 1)
    d = torch.randint(-far, far + 1, (N, groups, g), generator=gen)
    lo, hi = (-(1 << bits - 1), (1 << bits - 1) - 1) if sym else (0, (1 << bits) - 1)
    z = torch.zeros(N, groups) if sym else torch.randint(0, 1 << bits, (N, groups), generator=gen).float()
    q = (d + z[..., None].long()).clamp(lo, hi).view(N, K) & ((1 << bits) - 1)
    if bits == 4:
        q = q[:, 0::2] | (q[:, 1::2] << 4)
    return q.to(torch.uint8).cuda(), s.cuda(), z.bfloat16().cuda()


def one_hot(M, K):
    at = [(37 * m + 5) % K for m in range(M)]
    X = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    X[torch.arange(M), at] = 1.0
    return X, at


EXPONENTS = [-120, -60, 60, 118, 121, 122, 124, 126]


@pytest.mark.parametrize("exponent", EXPONENTS)
@pytest.mark.parametrize("M", [1, 8, 13])
@pytest.mark.parametrize("g", [32, 64, 128, 0])
@pytest.mark.parametrize("sym", [False, True])
def test_gemm8(exponent, M, g, sym):
    N, K = 300, 1152
    w = weights(N, K, g or K, 8, sym, exponent, M)
    W = w4.dequantize8(*w, g=g or K, sym=sym)
    assert bool(W.isfinite().all())
    X, at = one_hot(M, K)
    for path in ("decode", "tensorcore"):
        assert torch.equal(w4.gemm8(X, *w, g=g or K, sym=sym, path=path), W[:, at].t()), path


@pytest.mark.parametrize("exponent", EXPONENTS)
@pytest.mark.parametrize("M", [1, 8, 13])
@pytest.mark.parametrize("g", [32, 128, 0])
@pytest.mark.parametrize("bits,sym", [(4, False), (4, True), (8, False), (8, True)])
def test_gated_decode(exponent, M, g, bits, sym):
    N, K = 300, 1152
    gate, up = weights(N, K, g or K, bits, sym, exponent, M), weights(N, K, g or K, bits, sym, exponent, M + 50)
    f, dq = (w4.gated, w4.dequantize) if bits == 4 else (w4.gated8, w4.dequantize8)
    X, at = one_hot(M, K)
    _, G, U = f(X, gate, up, g=g or K, sym=sym, act="relu", save=True, path="decode")
    for Y, w in ((G, gate), (U, up)):
        W = dq(*w, g=g or K, sym=sym)
        assert bool(W.isfinite().all())
        assert torch.equal(Y, W[:, at].t())


TAKEN = [e for e in EXPONENTS if e < 122]


@pytest.mark.parametrize("exponent", EXPONENTS)
@pytest.mark.parametrize("M", [40, 90, 200])
@pytest.mark.parametrize("g", [32, 64, 128, 0])
@pytest.mark.parametrize("bits,sym", [(4, False), (4, True), (8, False), (8, True)])
def test_gated_tensor_cores(exponent, M, g, bits, sym):
    """Exact below 2^122; from there on the call says that it met such a scale."""
    N, K = 300, 1152
    gate, up = weights(N, K, g or K, bits, sym, exponent, M), weights(N, K, g or K, bits, sym, -5, M + 50)
    f, dq = (w4.gated, w4.dequantize) if bits == 4 else (w4.gated8, w4.dequantize8)
    X, at = one_hot(M, K)
    for a, b in ((gate, up), (up, gate)):
        _, G, U = f(X, a, b, g=g or K, sym=sym, act="relu", save=True)
        if exponent not in TAKEN:
            assert w4.device_error() == 4
            continue
        for Y, w in ((G, a), (U, b)):
            W = dq(*w, g=g or K, sym=sym)
            assert bool(W.isfinite().all())
            assert torch.equal(Y, W[:, at].t())


@pytest.mark.parametrize("exponent", EXPONENTS)
@pytest.mark.parametrize("N", [40, 300])
@pytest.mark.parametrize("g", [32, 64, 128, 0])
@pytest.mark.parametrize("bits,sym", [(4, False), (4, True), (8, False), (8, True)])
def test_gemm_dgrad(exponent, N, g, bits, sym):
    K = 1152
    w = weights(N, K, g or K, bits, sym, exponent, N)
    f, dq = (w4.gemm_dgrad, w4.dequantize) if bits == 4 else (w4.gemm8_dgrad, w4.dequantize8)
    W = dq(*w, g=g or K, sym=sym)
    assert bool(W.isfinite().all())
    eye = torch.eye(N, dtype=torch.bfloat16, device="cuda")
    for rows in (eye, eye[:17].contiguous()):
        dX = f(rows, *w, g=g or K, sym=sym)
        if exponent not in TAKEN:
            assert w4.device_error() == 4
        else:
            assert torch.equal(dX, W[:rows.shape[0]])


def test_one_wide_scale_is_enough():
    """Wherever it stands: first and last row, first and last group, gate or up, one product of two."""
    N, K, g, M = 300, 1152, 64, 40
    gate, up = weights(N, K, g, 4, False, -5, 1), weights(N, K, g, 4, False, -5, 2)
    X, _ = one_hot(M, K)
    dH = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    w4.gated(X, gate, up, g=g)
    w4.gated_backward(dH, dH, dH, gate, up, g=g)
    assert w4.device_error() == 0
    for n in (0, 131, N - 1):
        for j in (0, 7, K // g - 1):
            for which in range(2):
                pair = [gate, up]
                s = pair[which][1].clone()
                s[n, j] = 2.0 ** 122
                pair[which] = (pair[which][0], s, pair[which][2])
                w4.gated(X, *pair, g=g)
                assert w4.device_error() == 4
                w4.gated_backward(dH, dH, dH, *pair, g=g)
                assert w4.device_error() == 4
                w4.gemm_dgrad(dH, *pair[which], g=g)
                assert w4.device_error() == 4
                w4.gated(X[:8].contiguous(), *pair, g=g)      # the decode path takes it
                assert w4.device_error() == 0


@pytest.mark.parametrize("exponent", EXPONENTS)
@pytest.mark.parametrize("g", [32, 128, 0])
@pytest.mark.parametrize("bits,sym", [(4, False), (4, True), (8, False), (8, True)])
def test_embedding(exponent, g, bits, sym):
    V, K = 70, 1152
    w = weights(V, K, g or K, bits, sym, exponent, 9)
    f, dq = (w4.embedding, w4.dequantize) if bits == 4 else (w4.embedding8, w4.dequantize8)
    assert torch.equal(f(torch.arange(V, device="cuda"), *w, g=g or K, sym=sym), dq(*w, g=g or K, sym=sym))
