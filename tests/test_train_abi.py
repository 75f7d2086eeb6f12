"""Refusals of the gated block, the gradients and the embedding, at the C ABI and at the
binding: nothing here launches a kernel, and no GPU is needed."""
import ctypes

import pytest
import torch

import weight_only_quantization_rtn_b200 as w4
from weight_only_quantization_rtn_b200 import build as w4build

EINVAL, EWORKSPACE = 1, 4
P = ctypes.c_void_p(0x10000)        # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p(0x10008)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    w4build.build()
    return w4.lib()


def gated(lib, bits=4, X=P, M=4, K=256, w=(P, P, P), u=(P, P, P), N=64, g=128, sym=0, act=0, H=P, G=None, U=None,
          ws=P, wb=BIG, path=0):
    f = lib.w4a16_gated if bits == 4 else lib.w8a16_gated
    return f(X, M, K, *w, *u, N, g, sym, act, H, G, U, ws, wb, path, None)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("bad", [dict(K=250), dict(K=0), dict(g=96), dict(g=0), dict(M=-1), dict(N=-1), dict(sym=2),
                                 dict(act=4), dict(act=-1), dict(X=None), dict(H=None), dict(X=ODD), dict(H=ODD),
                                 dict(w=(None, P, P)), dict(w=(P, None, P)), dict(w=(P, P, None)), dict(u=(P, P, None)),
                                 dict(u=(P, ODD, P)), dict(G=P), dict(U=P), dict(G=P, U=ODD), dict(ws=None),
                                 dict(ws=ODD), dict(path=3), dict(path=1, M=17), dict(N=1 << 31), dict(M=1 << 31)])
def test_gated_refuses(lib, bits, bad):
    assert gated(lib, bits, **bad) == EINVAL


def test_gated_small_workspace_and_empty(lib):
    need = lib.w4a16_gated_workspace_size(4, 64, 256, 128, 0)
    assert need > 0 and gated(lib, wb=need - 1) == EWORKSPACE
    need = lib.w4a16_gated_workspace_size(40, 64, 4096, 128, 0)
    assert need > 0 and gated(lib, M=40, K=4096, wb=need - 1) == EWORKSPACE
    assert gated(lib, M=0, X=None) == 0 and gated(lib, N=0, H=None) == 0
    assert lib.w4a16_gated_workspace_size(4, 64, 250, 128, 0) == 0
    assert lib.w4a16_gated_workspace_size(17, 64, 256, 128, 1) == 0


def gated_backward(lib, bits=4, dH=P, G=P, U=P, M=40, N=64, w=(P, P, P), u=(P, P, P), K=256, g=128, sym=0, act=0, dX=P,
                   dG=P, dU=P, ws=P, wb=BIG):
    f = lib.w4a16_gated_backward if bits == 4 else lib.w8a16_gated_backward
    return f(dH, G, U, M, N, *w, *u, K, g, sym, act, dX, dG, dU, ws, wb, None)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("bad", [dict(K=250), dict(g=96), dict(M=-1), dict(N=-1), dict(sym=-1), dict(act=9),
                                 dict(dH=None), dict(G=None), dict(U=None), dict(dX=None), dict(dG=None), dict(dU=None),
                                 dict(dG=ODD), dict(dX=ODD), dict(w=(P, P, None)), dict(u=(None, P, P)),
                                 dict(N=63, ws=None), dict(N=63, ws=ODD)])
def test_gated_backward_refuses(lib, bits, bad):
    assert gated_backward(lib, bits, **bad) == EINVAL


def test_gated_backward_workspace(lib):
    # rows of 63 are padded to 64: two copies of 40 rows, 256-byte multiples
    need = lib.w4a16_gated_backward_workspace_size(40, 63, 256, 128)
    assert need == 2 * 40 * 64 * 2
    assert gated_backward(lib, N=63, wb=need - 1) == EWORKSPACE
    assert gated_backward(lib, M=0, dX=None) == 0


@pytest.mark.parametrize("f", ["w4a16_gemm_dgrad", "w8a16_gemm_dgrad"])
def test_dgrad_refuses(lib, f):
    def call(dY=P, M=40, N=64, w=(P, P, P), K=256, g=128, sym=0, dX=P, ws=P, wb=BIG):
        return getattr(lib, f)(dY, M, N, *w, K, g, sym, dX, ws, wb, None)
    for bad in (dict(K=250), dict(g=1), dict(M=-1), dict(N=-1), dict(sym=3), dict(dY=None), dict(dX=None),
                dict(dY=ODD), dict(w=(P, P, None)), dict(w=(ODD, P, P)), dict(N=63, ws=None)):
        assert call(**bad) == EINVAL, bad
    assert call(N=63, wb=lib.w4a16_gemm_dgrad_workspace_size(40, 63, 256, 128) - 1) == EWORKSPACE
    assert call(M=0, dX=None) == 0


def test_wgrad_refuses(lib):
    def call(dY=P, X=P, M=40, N=64, K=256, dW=P, ws=P, wb=BIG):
        return lib.w4a16_gemm_wgrad(dY, X, M, N, K, dW, ws, wb, None)
    for bad in (dict(K=40), dict(K=0), dict(M=-1), dict(N=-1), dict(dY=None), dict(X=None), dict(dW=None), dict(X=ODD),
                dict(dW=ODD), dict(N=63, ws=None), dict(M=1 << 31)):
        assert call(**bad) == EINVAL, bad
    assert call(N=63, wb=40 * 64 * 2 - 1) == EWORKSPACE
    assert call(N=0, dW=None) == 0


@pytest.mark.parametrize("f", ["w4a16_embedding", "w8a16_embedding"])
def test_embedding_refuses(lib, f):
    def call(ids=P, ib=8, T=4, w=(P, P, P), V=64, K=256, g=128, sym=0, out=P):
        return getattr(lib, f)(ids, ib, T, *w, V, K, g, sym, 1.0, out, None)
    for bad in (dict(K=250), dict(g=5), dict(T=-1), dict(V=-1), dict(ib=2), dict(ids=None), dict(out=None), dict(out=ODD),
                dict(w=(P, P, None)), dict(w=(None, P, P)), dict(sym=2)):
        assert call(**bad) == EINVAL, bad
    assert call(T=0, ids=None) == 0


def test_embedding_grad_refuses(lib):
    def call(dY=P, ids=P, ib=8, T=40, V=64, K=256, f32=1, dW=P, ws=P, wb=BIG):
        return lib.w4a16_embedding_grad(dY, ids, ib, T, V, K, 1.0, f32, dW, ws, wb, None)
    for bad in (dict(K=20), dict(K=0), dict(T=-1), dict(V=-1), dict(ib=1), dict(f32=2), dict(dY=None), dict(ids=None),
                dict(dW=None), dict(dW=ODD), dict(ws=None), dict(ws=ODD), dict(T=1 << 31), dict(V=(1 << 31) - 1)):
        assert call(**bad) == EINVAL, bad
    need = lib.w4a16_embedding_grad_workspace_size(40, 64, 256)
    assert call(wb=need - 1) == EWORKSPACE
    assert call(V=0, dW=None) == 0
    assert lib.w4a16_embedding_grad_workspace_size(0, 64, 256) == 0


def test_binding_refuses_before_the_call():
    """Host tensors, wrong types and shapes raise in the binding."""
    bf, u8 = torch.bfloat16, torch.uint8
    X, dY = torch.zeros(4, 256, dtype=bf), torch.zeros(4, 64, dtype=bf)
    w = (torch.zeros(64, 128, dtype=u8), torch.zeros(64, 2, dtype=bf), torch.zeros(64, 2, dtype=bf))
    with pytest.raises(ValueError):
        w4.gated(X, w, w)                                   # not on a CUDA device
    with pytest.raises(TypeError):
        w4.gated(X.float(), w, w)
    with pytest.raises(ValueError):
        w4.gated_backward(dY, dY, dY, w, w)
    with pytest.raises(ValueError):
        w4.gemm_dgrad(dY, *w)
    with pytest.raises(TypeError):
        w4.gemm_wgrad(dY.half(), X)
    with pytest.raises(ValueError):
        w4.gemm_wgrad(dY, X)
    with pytest.raises(TypeError):
        w4.embedding(X, *w)
    with pytest.raises(ValueError):
        w4.embedding(torch.zeros(3, dtype=torch.int64), *w)
    with pytest.raises(TypeError):
        w4.embedding_grad(dY, torch.zeros(4, dtype=torch.int16), 10)
    with pytest.raises(ValueError):
        w4.embedding_grad(dY, torch.zeros(4, dtype=torch.int64), 10)
