"""Cases of the operators around the quantized linear layer: the gated feed-forward
block and its backward pass, the linear layer's gradients, and the quantized
embedding with its table's gradient.

Each case is one pass of one operator on the GPU.  With ``own`` false ``run``
computes the operator's plain form in binary32 from elementary torch operations;
with ``own`` true it makes the calls a user makes of this package.

Weights are W[N, K] quantized by rounding to the nearest (4-bit codes two per byte,
or 8-bit codes), with one bf16 scale and zero point per group of g input channels
(g = 0 in a case: one group per row).  The weight they stand for is
bf16((q - z)*s).  Shapes follow the 7B- and 70B-shaped feed-forward layers and the
square layer of this repository's workloads; the vocabulary is a generic 32000 rows.
"""
import math

import torch

own = False
DEV = "cuda"
BF16 = torch.bfloat16


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token of a decode step through the feed-forward block of the 7B-shaped model
        dict(name="gated_m1", op="gated", M=1, K=4096, N=11008, bits=4, g=128, sym=False,
             act="silu", save=False),
        # eight sequences decoded together, the 70B-shaped block, symmetric codes
        dict(name="gated_m8_70b", op="gated", M=8, K=8192, N=28672, bits=4, g=128, sym=True,
             act="silu", save=False),
        # a ragged batch of short prompts, finer groups
        dict(name="gated_m61", op="gated", M=61, K=4096, N=11008, bits=4, g=64, sym=False,
             act="gelu_tanh", save=False),
        # a training (or prefill) step's tokens, both projections kept for the backward pass
        dict(name="gated_m2048_save", op="gated", M=2048, K=4096, N=11008, bits=4, g=128,
             sym=False, act="silu", save=True),
        # the backward pass of that step
        dict(name="gated_bwd_m2048", op="gated_backward", M=2048, K=4096, N=11008, bits=4, g=128,
             sym=False, act="silu"),
        # a small ragged micro-batch on 8-bit codes with one scale per row
        dict(name="gated_bwd_m333_w8", op="gated_backward", M=333, K=4096, N=11008, bits=8, g=0,
             sym=True, act="gelu"),
        # gradients of the 7B-shaped down projection at a training step's tokens
        dict(name="linear_bwd_m2048", op="linear_backward", M=2048, K=11008, N=4096, bits=4,
             g=128, sym=False),
        # a square layer with a short ragged micro-batch
        dict(name="linear_bwd_m77", op="linear_backward", M=77, K=8192, N=8192, bits=4, g=128,
             sym=True),
        # the embedding of a decode step's tokens
        dict(name="embed_t16", op="embedding", T=16, V=32000, K=4096, bits=4, g=128, sym=False,
             scale=1.0),
        # the embedding of a long prompt or training batch, 8-bit table, scaled by sqrt(K)
        dict(name="embed_t8192_w8", op="embedding", T=8192, V=32000, K=8192, bits=8, g=128,
             sym=False, scale=math.sqrt(8192.0)),
        # the table's gradient for one sequence of 2048 tokens, some of them padding
        dict(name="embed_grad_t2048", op="embedding_grad", T=2048, V=32000, K=4096,
             dtype="bfloat16", scale=1.0, pad=True),
        # and for a batch of 16384 tokens, kept in binary32
        dict(name="embed_grad_t16384", op="embedding_grad", T=16384, V=32000, K=4096,
             dtype="float32", scale=64.0, pad=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_backward", "linear_backward", "embedding",
                     "embedding_grad"])
    bits, g, sym = rng.choice([4, 4, 8]), rng.choice([32, 64, 128, 128, 0]), rng.random() < 0.5
    step = g if g else 32
    if op in ("embedding", "embedding_grad"):
        K = max(1, _log(rng, 256, 8192) // step) * step
        T, V = _log(rng, 1, 16384), _log(rng, 300, 48000)
        if op == "embedding":
            return dict(op=op, T=T, V=V, K=K, bits=bits, g=g, sym=sym,
                        scale=rng.choice([1.0, 0.5, math.sqrt(K)]))
        K = min(K, 4096)
        return dict(op=op, T=T, V=min(V, 32000), K=K, dtype=rng.choice(["bfloat16", "float32"]),
                    scale=rng.choice([1.0, math.sqrt(K)]), pad=rng.random() < 0.5)
    M = _log(rng, 1, 2048)
    if op == "gated" and rng.random() < 0.4:
        M = rng.randint(1, 16)
    K = max(1, _log(rng, 256, 8192) // step) * step
    N = _log(rng, 128, 11008)
    if M > 1024:
        K = min(K, 4096)
    c = dict(op=op, M=M, K=K, N=N, bits=bits, g=g, sym=sym)
    if op != "linear_backward":
        c["act"] = rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"])
    if op == "gated":
        c["save"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------- inputs
def _quantized(gen, N, K, bits, g, sym, sigma=0.02):
    """Codes, scales and zero points of a normal weight, by rounding to the nearest."""
    g = g or K
    W = (torch.randn(N, K, generator=gen, device=DEV) * sigma).to(BF16).float().view(N, K // g, g)
    if sym:
        s = (W.abs().amax(2) / (7 if bits == 4 else 127)).to(BF16)
        z = torch.zeros_like(s)
        lo, hi = (-8, 7) if bits == 4 else (-128, 127)
    else:
        lo, hi = 0, 15 if bits == 4 else 255
        mn, mx = W.amin(2).clamp(max=0), W.amax(2).clamp(min=0)
        s = ((mx - mn) / hi).to(BF16)
        z = (-mn / s.float()).round().clamp(0, hi).to(BF16)
    q = ((W / s.float()[..., None]).round() + z.float()[..., None]).clamp(lo, hi)
    q = q.view(N, K).to(torch.int16)
    if bits == 8:
        return (q & 255).to(torch.uint8), s, z
    q = q & 15
    return (q[:, 0::2] | (q[:, 1::2] << 4)).to(torch.uint8).contiguous(), s, z


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    c, st = case, {"case": case}

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device=DEV) * std).to(BF16)

    if c["op"] in ("embedding", "embedding_grad"):
        # ids with the long tail of text: a few rows take most tokens
        u = torch.rand(c["T"], generator=gen, device=DEV, dtype=torch.float64)
        ids = ((c["V"] ** u) - 1.0).long().clamp(0, c["V"] - 1)
        ids = (ids * 7919) % c["V"]
        if c.get("pad"):
            # sequences are padded at their end: an id below zero is no token
            ids[c["T"] - c["T"] // 8:] = -1
        st["ids"] = ids
        if c["op"] == "embedding":
            st["w"] = _quantized(gen, c["V"], c["K"], c["bits"], c["g"], c["sym"])
        else:
            st["dY"] = normal(c["T"], c["K"], std=0.01)
        return st
    M, N, K = c["M"], c["N"], c["K"]
    if c["op"] == "linear_backward":
        st["w"] = _quantized(gen, N, K, c["bits"], c["g"], c["sym"])
        st["X"], st["dY"] = normal(M, K), normal(M, N, std=0.01)
        return st
    st["gate"] = _quantized(gen, N, K, c["bits"], c["g"], c["sym"])
    st["up"] = _quantized(gen, N, K, c["bits"], c["g"], c["sym"])
    if c["op"] == "gated":
        st["X"] = normal(M, K)
    else:
        st["dH"], st["G"], st["U"] = normal(M, N, std=0.01), normal(M, N, std=1.3), normal(M, N, std=1.3)
    return st


# ---------------------------------------------------------------- plain forms (binary32)
def _codes(w, bits, sym):
    q = w.to(torch.int16)
    if bits == 4:
        q = torch.stack((q & 15, q >> 4), dim=-1).flatten(-2)
    if sym:
        half = 8 if bits == 4 else 128
        q = torch.where(q >= half, q - 2 * half, q)
    return q


def _weight(w, c):
    """bf16((q - z)*s), held in binary32."""
    codes, s, z = w
    q = _codes(codes, c["bits"], c["sym"]).float()
    N, K = q.shape
    g = c["g"] or K
    q = q.view(N, K // g, g) - z.float()[..., None]
    return (q * s.float()[..., None]).to(BF16).float().view(N, K)


def _act(x, kind):
    """The activation and its derivative."""
    if kind == "silu":
        p = 1 / (1 + torch.exp(-x))
        return x * p, p * (1 + x * (1 - p))
    if kind == "relu":
        return torch.where(x > 0, x, 0 * x), (x > 0).float()
    if kind == "gelu":
        p = 0.5 * (1 + torch.erf(x * math.sqrt(0.5)))
        return x * p, p + x * torch.exp(-0.5 * x * x) * (1 / math.sqrt(2 * math.pi))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (x + 0.044715 * x * x * x))
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * k * (1 + 0.134145 * x * x)


def _plain(st):
    c = st["case"]
    if c["op"] == "embedding":
        ids, (codes, s, z) = st["ids"], st["w"]
        return (_weight((codes[ids], s[ids], z[ids]), c) * c["scale"]).to(BF16)
    if c["op"] == "embedding_grad":
        d = torch.zeros(c["V"] + 1, c["K"], device=DEV)
        at = torch.where(st["ids"] < 0, c["V"], st["ids"])
        d.index_add_(0, at, st["dY"].float())
        return (d[:-1] * c["scale"]).to(getattr(torch, c["dtype"]))
    if c["op"] == "gated":
        X = st["X"].float()
        G, U = X @ _weight(st["gate"], c).t(), X @ _weight(st["up"], c).t()
        H = (_act(G, c["act"])[0] * U).to(BF16)
        return (H, G.to(BF16), U.to(BF16)) if c["save"] else H
    if c["op"] == "gated_backward":
        dH, G, U = st["dH"].float(), st["G"].float(), st["U"].float()
        a, da = _act(G, c["act"])
        dG, dU = dH * U * da, dH * a
        dX = dG @ _weight(st["gate"], c) + dU @ _weight(st["up"], c)
        return dX.to(BF16), dG.to(BF16), dU.to(BF16)
    dY = st["dY"].float()
    return (dY @ _weight(st["w"], c)).to(BF16), (dY.t() @ st["X"].float()).to(BF16)


# ---------------------------------------------------------------- the package's calls
def _own(st):
    import weight_only_quantization_rtn_b200 as w4
    c = st["case"]
    eight = c.get("bits") == 8
    if c["op"] == "embedding_grad":
        return w4.embedding_grad(st["dY"], st["ids"], c["V"], scale=c["scale"],
                                 dtype=getattr(torch, c["dtype"]))
    g, sym = c["g"] or c["K"], c["sym"]
    if c["op"] == "embedding":
        f = w4.embedding8 if eight else w4.embedding
        return f(st["ids"], *st["w"], g=g, sym=sym, scale=c["scale"])
    if c["op"] == "gated":
        f = w4.gated8 if eight else w4.gated
        return f(st["X"], st["gate"], st["up"], g=g, sym=sym, act=c["act"], save=c["save"])
    if c["op"] == "gated_backward":
        f = w4.gated8_backward if eight else w4.gated_backward
        return f(st["dH"], st["G"], st["U"], st["gate"], st["up"], g=g, sym=sym, act=c["act"])
    f = w4.gemm8_dgrad if eight else w4.gemm_dgrad
    return f(st["dY"], *st["w"], g=g, sym=sym), w4.gemm_wgrad(st["dY"], st["X"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without
def _weight_bytes(N, K, c):
    groups = N * (K // (c["g"] or K))
    return N * K * c["bits"] // 8 + groups * (2 if c["sym"] else 4)


def work(case):
    c = case
    if c["op"] == "embedding":
        row = c["K"] * c["bits"] // 8 + (c["K"] // (c["g"] or c["K"])) * (2 if c["sym"] else 4)
        return {"bytes": c["T"] * (8 + 2 * c["K"] + row), "flops": 3 * c["T"] * c["K"]}
    if c["op"] == "embedding_grad":
        e = 4 if c["dtype"] == "float32" else 2
        return {"bytes": c["T"] * (8 + 2 * c["K"]) + c["V"] * c["K"] * e,
                "flops": c["T"] * c["K"]}
    M, N, K = c["M"], c["N"], c["K"]
    if c["op"] == "gated":
        return {"bytes": 2 * _weight_bytes(N, K, c) + 2 * M * K + 2 * M * N * (3 if c["save"] else 1),
                "flops": 4 * M * N * K}
    if c["op"] == "gated_backward":
        return {"bytes": 2 * _weight_bytes(N, K, c) + 2 * M * K + 2 * M * N * 5,
                "flops": 4 * M * N * K}
    return {"bytes": _weight_bytes(N, K, c) + 2 * M * (2 * K + N) + 2 * N * K,
            "flops": 4 * M * N * K}


# ---------------------------------------------------------------- the definition in binary64
def _weight64(w, c):
    """The same weights by a table of each group's levels."""
    codes, s, z = w
    raw = codes.long()
    if c["bits"] == 4:
        raw = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.long, device=DEV)
        raw[:, 0::2], raw[:, 1::2] = codes.long() % 16, codes.long() // 16
    n = 1 << c["bits"]
    level = torch.arange(n, device=DEV, dtype=torch.float64)
    if c["sym"]:
        level = (level + n // 2) % n - n // 2
    W = torch.empty(raw.shape, dtype=torch.float64, device=DEV)
    g = c["g"] or raw.shape[1]
    for j in range(raw.shape[1] // g):
        table = ((level[None, :] - z[:, j:j + 1].double()) * s[:, j:j + 1].double()).to(BF16).double()
        W[:, j * g:(j + 1) * g] = torch.gather(table, 1, raw[:, j * g:(j + 1) * g])
    return W


def _act64(x, kind):
    if kind == "silu":
        return x * torch.sigmoid(x)
    if kind == "relu":
        return torch.clamp(x, min=0)
    if kind == "gelu":
        return 0.5 * x * torch.erfc(-x / math.sqrt(2.0))
    return x * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))


def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["op"] == "embedding":
        codes, s, z = st["w"]
        rows, back = torch.unique(st["ids"], return_inverse=True)
        return _weight64((codes[rows], s[rows], z[rows]), c)[back] * c["scale"]
    if c["op"] == "embedding_grad":
        out = torch.zeros(c["V"], c["K"], dtype=torch.float64, device=DEV)
        keep = (st["ids"] >= 0).nonzero()[:, 0]
        out.index_put_((st["ids"][keep],), st["dY"][keep].double() * c["scale"], accumulate=True)
        return out
    if c["op"] == "linear_backward":
        dY = st["dY"].double()
        return torch.mm(dY, _weight64(st["w"], c)), torch.mm(dY.t(), st["X"].double())
    if c["op"] == "gated":
        X = st["X"].double()
        G = torch.mm(_weight64(st["gate"], c), X.t()).t()
        U = torch.mm(_weight64(st["up"], c), X.t()).t()
        H = _act64(G, c["act"]) * U
        return (H, G, U) if c["save"] else H
    G = st["G"].double().requires_grad_(True)
    a = _act64(G, c["act"])
    dG, = torch.autograd.grad(a.sum(), G)
    dH = st["dH"].double()
    dG, dU = dG * dH * st["U"].double(), a.detach() * dH
    return torch.mm(dG, _weight64(st["gate"], c)) + torch.mm(dU, _weight64(st["up"], c)), dG, dU
