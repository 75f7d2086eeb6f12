"""The block, its gradients and the embedding where their paths change or their indexes are
largest: extreme scales and activations, offsets past 2^31, long id lists and tables,
work shared by many CTAs on several streams at once, ids at any address, in-place gradients."""
import pytest
import torch

import workloads
import weight_only_quantization_rtn_b200 as w4
from weight_only_quantization_rtn_b200 import build as w4build
from helpers import assert_y_close
from test_gpu_gated import act64, quantized

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    w4build.build()
    yield
    assert w4.device_error() == 0


def random_weights(N, K, g, bits, seed):
    """Codes drawn on the device (no dense weight exists), zeros 0 .. 15 or 0 .. 255."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (N, K * bits // 8), generator=gen, dtype=torch.uint8, device="cuda")
    scales = (torch.rand(N, K // g, generator=gen, device="cuda") * 0.02 + 0.001).bfloat16()
    zeros = torch.randint(0, 1 << bits, (N, K // g), generator=gen, device="cuda").bfloat16()
    return codes, scales, zeros


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M", [40, 200])
@pytest.mark.parametrize("exponent", [-110, -60, 60, 118])
def test_extreme_scales_are_exact(bits, M, exponent):
    """Identity rows return Ŵ bit for bit while s < 2^122 and |Ŵ| is a normal bf16 number."""
    N, K, g = M, 320, 64
    gen = torch.Generator().manual_seed(exponent + 200)
    codes, _, zeros = random_weights(N, K, g, bits, 5)
    s = torch.ldexp(1 + torch.rand(N, K // g, generator=gen), torch.tensor(exponent)).bfloat16().cuda()
    if exponent == 118:
        s = s * (1.0 if bits == 4 else 2.0 ** -4)                # |q − z|·s < 2^127
    dq, f, emb = ((w4.dequantize, w4.gemm_dgrad, w4.embedding) if bits == 4 else
                  (w4.dequantize8, w4.gemm8_dgrad, w4.embedding8))
    W = dq(codes, s, zeros, g=g)
    assert bool(W.isfinite().all())
    eye = torch.eye(N, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(f(eye, codes, s, zeros, g=g), W)
    assert torch.equal(emb(torch.arange(N, device="cuda"), codes, s, zeros, g=g), W)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("N", [64, 65])
def test_gate_gradient_of_extreme_projections(act, N):
    """Far out every activation is 0 or x and its derivative 0 or 1; at 0 they are exact."""
    vals = [0.0, 1e-30, -1e-30, 8.0, -40.0, 40.0, -1e4, 1e4, 1e10, -1e10, 1e20, -1e20, 1e38, -1e38]
    G = torch.tensor(vals, dtype=torch.bfloat16, device="cuda")[:, None].expand(len(vals), N).contiguous()
    dH, U = torch.full_like(G, 0.5), torch.full_like(G, 0.25)
    w, _ = quantized(N, 32, 32, False, 4, 3)
    _, dG, dU = w4.gated_backward(dH, G, U, w, w, g=32, act=act)
    x = G.double().requires_grad_(True)
    a = act64(x, act)
    d, = torch.autograd.grad(a.sum(), x)
    a = a.detach()
    if act == "gelu_tanh":                       # (automatic differentiation multiplies 0 by x²'s infinity)
        d = torch.where(d.isnan(), (x > 0).double(), d).detach()
    assert bool(dG.isfinite().all() and dU.isfinite().all())
    # one rounding to bf16 (2^-8 relative), 2^-20 of the arithmetic before it, and what of the
    # exponential tail lies below binary32's normal range
    for got, want in ((dG, 0.5 * 0.25 * d), (dU, 0.5 * a)):
        assert bool(((got.double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -12) + 2.0 ** -40).all()), act


def test_in_place_gate_gradient():
    """dG and dU may take G's and U's own memory (rows of 8 and odd rows)."""
    L = w4.lib()
    for M, N, K in ((33, 128, 64), (5, 77, 96), (300, 256, 64)):
        g = 32
        w, _ = quantized(N, K, g, False, 4, 7)
        dH, G, U = (workloads.make_activation(M, N, s).cuda() for s in (1, 2, 3))
        want = w4.gated_backward(dH, G, U, w, w, g=g)
        dX = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
        nbytes = L.w4a16_gated_backward_workspace_size(M, N, K, g)
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda")
        ptrs = [t.data_ptr() for t in w]
        assert L.w4a16_gated_backward(dH.data_ptr(), G.data_ptr(), U.data_ptr(), M, N, *ptrs, *ptrs, K, g, 0, 0,
                                      dX.data_ptr(), G.data_ptr(), U.data_ptr(), ws.data_ptr(), nbytes,
                                      torch.cuda.current_stream().cuda_stream) == 0
        assert all(torch.equal(a, b) for a, b in zip(want, (dX, G, U)))


def test_many_sharers_on_streams_and_in_graphs():
    """Tiles shared by several CTAs (few tiles, long reductions), three calls in flight at once,
    eager and as replayed graphs, give what one call gives, and the same bits each time."""
    N, K, g = 4096, 512, 128
    gate, Wg = quantized(N, K, g, False, 4, 51)
    up, Wu = quantized(N, K, g, True, 4, 52)
    up = (up[0], up[1], gate[2])                   # any zeros: asymmetric
    Wu = w4.dequantize(*up, g=g).double()
    Ms = (20, 90, 230)
    ins = [tuple(workloads.make_activation(M, N, 60 + 3 * i + j).cuda() for j in range(3)) for i, M in enumerate(Ms)]
    want = [w4.gated_backward(*t, gate, up, g=g) for t in ins]
    for (dX, dG, dU), M in zip(want, Ms):
        assert_y_close(workloads.bits(dX), (dG.double() @ Wg + dU.double() @ Wu).cpu().numpy(), f"M={M}")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Ms]
    got = []
    for _ in range(5):
        for s, t in zip(streams, ins):
            with torch.cuda.stream(s):
                got.append(w4.gated_backward(*t, gate, up, g=g))
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(r, want[i % 3]))
    graphs = []
    for t in ins:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o = w4.gated_backward(*t, gate, up, g=g)
        graphs.append((graph, o))
    for _ in range(5):
        for s, (graph, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (_, o), r in zip(graphs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, r))


@pytest.mark.parametrize("T,V,K,kind", [(40000, 5000, 64, "uniform"), (70000, 300, 32, "uniform"), (100000, 7, 32, "uniform"),
                                        (300, 5000000, 32, "uniform"), (70000, 5000000, 32, "uniform"),
                                        (131073, 40000, 64, "same")])
def test_embedding_grad_long_lists_and_tables(T, V, K, kind):
    """More ids than one shared-memory ranking takes, chunks of 16384, and keys of more than
    22 bits.  n additions are off by n·2^-24·Σ|dY| at most, the result by 2^-24."""
    gen = torch.Generator().manual_seed(T + V)
    ids = (torch.full((T,), V - 1) if kind == "same" else torch.randint(0, V, (T,), generator=gen)).cuda()
    ids[T // 3::11] = -1
    dY = workloads.make_activation(T, K, 8).cuda()
    out = torch.full((V, K), float("nan"), device="cuda")
    dW = w4.embedding_grad(dY, ids, V, out=out)
    keep = ids >= 0
    rows = ids[keep].unique()
    at = torch.searchsorted(rows, ids[keep])
    want = torch.zeros(len(rows), K, dtype=torch.float64, device="cuda").index_add_(0, at, dY[keep].double())
    mag = torch.zeros_like(want).index_add_(0, at, dY[keep].double().abs())
    n = torch.zeros(len(rows), dtype=torch.float64, device="cuda").index_add_(0, at, torch.ones_like(at).double())
    assert bool(((dW[rows].double() - want).abs() <= mag * (n[:, None] + 1) * 2.0 ** -24 + want.abs() * 2.0 ** -24).all())
    dW[rows] = 0
    assert bool((dW == 0).all())                    # the rest is zeros, and nothing was left unwritten
    assert torch.equal(w4.embedding_grad(dY, ids, V)[rows], w4.embedding_grad(dY, ids.int(), V)[rows])


def test_ids_at_any_address():
    w = w4.quantize(workloads.make_weight(50, 64, 0.02, 1).cuda(), 64, False)
    ids = torch.randint(0, 50, (41,), generator=torch.Generator().manual_seed(1)).cuda()
    dY = workloads.make_activation(41, 64, 2).cuda()
    for dt in (torch.int64, torch.int32):
        part = ids.to(dt)[3:]
        assert torch.equal(w4.embedding(part, *w, g=64), w4.embedding(part.clone(), *w, g=64))
        assert torch.equal(w4.embedding_grad(dY[3:], part, 50), w4.embedding_grad(dY[3:], part.clone(), 50))


def test_refusals_and_given_outputs():
    N, K, M = 96, 64, 20
    w, W = quantized(N, K, 32, False, 4, 1)
    X, dY = workloads.make_activation(M, K, 2).cuda(), workloads.make_activation(M, N, 3).cuda()
    ids = torch.arange(M, device="cuda")
    calls = {"gated": lambda **k: w4.gated(X, w, w, g=32, **k), "dgrad": lambda **k: w4.gemm_dgrad(dY, *w, g=32, **k),
             "wgrad": lambda **k: w4.gemm_wgrad(dY, X, **k), "embedding": lambda **k: w4.embedding(ids, *w, g=32, **k),
             "grad": lambda **k: w4.embedding_grad(X, ids, N, dtype=torch.bfloat16, **k),
             "backward": lambda **k: w4.gated_backward(dY, dY, dY, w, w, g=32, **k)[0]}
    for name, f in calls.items():
        want = f()
        out = torch.full_like(want, float("nan"))
        assert f(out=out).data_ptr() == out.data_ptr() and torch.equal(out, want), name
        wide = torch.empty(want.shape[0], 2 * want.shape[1], dtype=torch.bfloat16, device="cuda")
        for bad, error in ((out.float(), TypeError), (out.cpu(), ValueError), (out[1:], ValueError),
                           (wide[:, ::2], ValueError)):
            with pytest.raises(error):
                f(out=bad)
    strided = workloads.make_activation(M, 2 * K, 2).cuda()[:, ::2]
    for f in (lambda: w4.gated(strided, w, w, g=32), lambda: w4.gemm_wgrad(dY, strided),
              lambda: w4.gemm_dgrad(dY.t(), *w, g=32), lambda: w4.embedding(ids[::2], *w, g=32),
              lambda: w4.embedding_grad(strided, ids, N), lambda: w4.gated(X, w, w, g=32, act="swish"),
              lambda: w4.gated(X, w, w, g=64), lambda: w4.embedding_grad(X, ids, -1)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(w4.W4A16Error):
        w4.gated(X, w, w, g=32, path="decode")             # more than 16 tokens


def test_offsets_past_31_bits():
    """Outputs, codes and rows whose element offsets need more than 31 bits."""
    M, N, K, g = 140000, 16384, 64, 64                        # M·N = 2.29e9
    gate, up = random_weights(N, K, g, 4, 1), random_weights(N, K, g, 4, 2)
    X = workloads.make_activation(M, K, 3).cuda()
    H, G, U = w4.gated(X, gate, up, g=g, save=True)
    dX, dG, dU = w4.gated_backward(G, H, U, gate, up, g=g)
    Wg, Wu = w4.dequantize(*gate, g=g).double(), w4.dequantize(*up, g=g).double()
    for m in (0, 131060, M - 40):                             # 131072 rows of 16384 are 2^31
        r = slice(m, m + 40)
        G64, U64 = X[r].double() @ Wg.t(), X[r].double() @ Wu.t()
        for got, want in ((G[r], G64), (U[r], U64), (H[r], act64(G64, "silu") * U64),
                          (dX[r], dG[r].double() @ Wg + dU[r].double() @ Wu)):
            assert_y_close(workloads.bits(got), want.cpu().numpy(), f"rows {m}")
        h = H[r].double()
        assert_y_close(workloads.bits(dU[r]), (G[r].double() * act64(h, "silu")).cpu().numpy(), f"dU rows {m}")
    del H, G, U, dX, dG, dU
    w = random_weights(64, N, 64, 4, 4)                       # dX [M, 16384]
    dY = workloads.make_activation(M, 64, 5).cuda()
    dX = w4.gemm_dgrad(dY, *w, g=64)
    W = w4.dequantize(*w, g=64).double()
    for m in (0, 131060, M - 40):
        assert_y_close(workloads.bits(dX[m:m + 40]), (dY[m:m + 40].double() @ W).cpu().numpy(), f"rows {m}")
    del dX, dY
    dY, X = workloads.make_activation(40, M, 6).cuda(), workloads.make_activation(40, N, 7).cuda()
    dW = w4.gemm_wgrad(dY, X)                                 # [140000, 16384]
    for m in (0, 131060, M - 40):
        assert_y_close(workloads.bits(dW[m:m + 40]), (dY[:, m:m + 40].double().t() @ X.double()).cpu().numpy(),
                       f"rows {m}")
    del dW
    V, K, g = 1100000, 4096, 128                              # 4.5e9 codes
    table = random_weights(V, K, g, 4, 8)
    ids = torch.tensor([0, 524287, 524288, 1048575, 1048576, V - 1, 7], device="cuda")
    W = w4.dequantize(*(t[ids].contiguous() for t in table), g=g)
    assert torch.equal(w4.embedding(ids, *table, g=g), W)
    dT = w4.embedding_grad(W, ids, V, dtype=torch.bfloat16)
    assert torch.equal(dT[ids], W)
    dT[ids] = 0
    assert all(int(c.count_nonzero()) == 0 for c in dT.split(100000))


@pytest.mark.parametrize("bits,M", [(8, 1), (8, 9), (4, 8), (4, 16)])
def test_short_batches_of_large_matrices(bits, M):
    """Both sides of the size from which up to 16 tokens go to the tensor cores: the path chosen
    and the two that can be forced agree with the plain product."""
    K, g = 2048, 128
    for N in (49152, 49160):                                  # 96·2^20 weights, and more
        gate, up = random_weights(N, K, g, bits, 11), random_weights(N, K, g, bits, 12)
        X = workloads.make_activation(M, K, 13).cuda()
        f, dq = (w4.gated, w4.dequantize) if bits == 4 else (w4.gated8, w4.dequantize8)
        want = act64(X.double() @ dq(*gate, g=g).double().t(), "silu") * (X.double() @ dq(*up, g=g).double().t())
        for path in ("auto", "decode", "tensorcore"):
            H = f(X, gate, up, g=g, path=path)
            assert_y_close(workloads.bits(H), want.cpu().numpy(), f"{bits} {M} {N} {path}")
