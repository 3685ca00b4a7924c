"""Operators of training routed experts, and 8-bit activation checkpoints, as cases to measure.

``run`` computes a case in its plain form (elementary torch operations in 32 bits, rounded where the definitions
below round), or, where ``own`` is true, by the calls of this repository's package.  ``exact`` gives the same outputs
from the definitions in 64 bits.

A token t has k pairs f = t k + j, each with an expert e(f); X[f / div] is row f of an operand that has a row a pair
(div = 1) or a row a token (div = k).

  experts     Y[f] = bf16(X[f / div] W_e^T), W [E, N, K]; transposed: bf16(X[f / div] W_e), W [E, K, N]
  wgrad       dW[e] = bf16(sum over e's pairs f of dY[f / dy_div]^T X[f / x_div]), zeros for an expert without pairs;
              X bf16, or a checkpoint: e4m3 codes with a power-of-two scale per 128 of a row
  tn          C = bf16(A^T B), A [M, N], B [M, K] (a checkpoint or bf16)
  swiglu      H = (g, u) (bf16 or a checkpoint), G the gradient of the down product's input before the top-k weight w:
              a = silu(g) u;  dH = bf16(w G u silu'(g), w G silu(g));  A = bf16(w a);  dw = sum G a
  linear      Y = Q(X) Q(W)^T with e4m3 codes (kind "w8"), or X F(W)^T with INT4 groups of 32 (kind "int4");
              dX = Q(dY) Q(W), or dY F(W);  dW = dY^T Q(X), from the checkpoint that the forward left
  layer       the routed layer's step: out, and the gradients of X, the top-k weights and both stacks of experts
"""

import math

import torch

own = False

DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


# ----------------------------------------------------------------------------------------------------- the cases --

def listed():
    return [
        # a fine-tuning step's first expert product on a handful of tokens: latency
        dict(name="experts_few", op="experts", T=4, k=2, E=8, N=1024, K=1024, transposed=False, pairs=False, skew=0.0),
        # the same in a training batch, some experts hotter than others
        dict(name="experts_batch", op="experts", T=4096, k=8, E=64, N=4096, K=2048, transposed=False, pairs=False,
             skew=1.0),
        # the input gradient of the first product, sizes that end inside every tile
        dict(name="experts_dgrad", op="experts", T=2050, k=6, E=48, N=2056, K=2808, transposed=True, pairs=True,
             skew=1.0),
        # weight gradients of a short batch: bound by writing them
        dict(name="wgrad_short", op="wgrad", T=64, k=4, E=32, N=1408, K=2048, side="gate_up", codes=False, skew=0.0),
        # weight gradients of a training batch
        dict(name="wgrad_batch", op="wgrad", T=4096, k=8, E=32, N=4096, K=4096, side="gate_up", codes=False, skew=1.0),
        # the same from 8-bit checkpoints, ragged
        dict(name="wgrad_codes", op="wgrad", T=3001, k=4, E=24, N=2056, K=4112, side="gate_up", codes=True, skew=1.0),
        # a linear layer's weight gradient from its input's checkpoint
        dict(name="tn_codes", op="tn", M=2050, N=4096, K=5120, codes=True),
        # between the two expert products, backward, of a short batch
        dict(name="swiglu_few", op="swiglu", R=64, I=2048, codes=False, weights=True),
        # the same of a long one from checkpoints, odd rows and a last block of 80
        dict(name="swiglu_codes", op="swiglu", R=32775, I=2000, codes=True, weights=True),
        # a training step of a linear layer that keeps its input in 8 bits
        dict(name="linear_step", op="linear", kind="w8", M=4096, N=4096, K=4096),
        # a routed INT4 layer's step on few tokens
        dict(name="layer_few", op="layer", T=32, k=4, E=8, H=1024, I=512, int4=True, checkpoint=True, skew=0.0),
        # a routed layer's step in a training batch
        dict(name="layer_batch", op="layer", T=4096, k=8, E=32, H=4096, I=2048, int4=False, checkpoint=True, skew=1.0),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["experts", "experts", "wgrad", "wgrad", "tn", "swiglu", "linear", "layer"])
    if op == "tn":
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 16, 4096, 8), K=_log(rng, 16, 5120, 16),
                    codes=rng.random() < 0.5)
    if op == "swiglu":
        return dict(op=op, R=_log(rng, 1, 32768), I=_log(rng, 16, 2048, 16), codes=rng.random() < 0.5,
                    weights=rng.random() < 0.7)
    if op == "linear":
        return dict(op=op, kind=rng.choice(["w8", "int4"]), M=_log(rng, 1, 4096), N=_log(rng, 64, 4096, 16),
                    K=_log(rng, 64, 4096, 32))
    E = rng.choice([1, 4, 8, 16, 32, 64])
    k = rng.randint(1, min(8, E))
    skew = rng.choice([0.0, 1.0, 2.0])
    if op == "experts":
        return dict(op=op, T=_log(rng, 1, 4096), k=k, E=E, N=_log(rng, 64, 4096, 8), K=_log(rng, 64, 4096, 8),
                    transposed=rng.random() < 0.5, pairs=rng.random() < 0.5, skew=skew)
    if op == "wgrad":
        return dict(op=op, T=_log(rng, 1, 4096), k=k, E=E, N=_log(rng, 64, 4096, 8), K=_log(rng, 64, 4096, 16),
                    side=rng.choice(["gate_up", "down"]), codes=rng.random() < 0.5, skew=skew)
    return dict(op=op, T=_log(rng, 1, 2048), k=k, E=min(E, 32), H=_log(rng, 64, 4096, 32), I=_log(rng, 64, 2048, 32),
                int4=rng.random() < 0.5, checkpoint=rng.random() < 0.5, skew=skew)


def _cols(K):
    return 4 * ((K + 511) // 512)


def _rows_bytes(R, K, codes):
    return R * (K + _cols(K)) if codes else 2 * R * K


def work(case):
    c = case
    op = c["op"]
    if op == "tn":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": 2 * M * N + _rows_bytes(M, K, c["codes"]) + 2 * N * K, "flops": 2 * M * N * K}
    if op == "swiglu":
        R, I = c["R"], c["I"]
        b = _rows_bytes(R, 2 * I, c["codes"]) + 8 * R * I + (8 * R if c["weights"] else 0)
        return {"bytes": b, "flops": 20 * R * I}
    if op == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": 4 * M * K + 4 * N * K + 4 * M * N, "flops": 6 * M * N * K}
    P = c["T"] * c["k"]
    used = min(c["E"], P)
    if op == "experts":
        N, K = c["N"], c["K"]
        return {"bytes": 2 * (P if c["pairs"] else c["T"]) * K + 2 * used * N * K + 2 * P * N, "flops": 2 * P * N * K}
    if op == "wgrad":
        N, K = c["N"], c["K"]
        dy, x = (P, c["T"]) if c["side"] == "gate_up" else (c["T"], P)
        return {"bytes": 2 * dy * N + _rows_bytes(x, K, c["codes"]) + 2 * c["E"] * N * K, "flops": 2 * P * N * K}
    H, I = c["H"], c["I"]
    # X and dOut in, out and dX back; weights in, their gradients back
    return {"bytes": 8 * c["T"] * H + 6 * (used + c["E"]) * H * I + 12 * P, "flops": 18 * P * H * I}


# ---------------------------------------------------------------------------------------------------- the inputs --

def _gen(seed, stream):
    return torch.Generator(device=DEV).manual_seed(seed * 1000003 + stream)


def _normal(shape, seed, stream, sigma=1.0):
    return (torch.randn(shape, generator=_gen(seed, stream), device=DEV, dtype=F32) * sigma).to(BF16)


def _hidden(M, K, seed, stream):
    """Hidden states: N(0, 1) with one channel in 64 sixteen times as large."""
    x = _normal((M, K), seed, stream)
    big = torch.randperm(K, generator=_gen(seed, stream + 50), device=DEV)[: max(1, K // 64)]
    x[:, big] *= 16
    return x


def _weights(E, N, K, seed, stream):
    W = torch.empty((E, N, K), dtype=BF16, device=DEV)
    for e in range(E):
        W[e] = _normal((N, K), seed, stream + e, 0.02)
    return W


def _picks(T, E, k, skew, seed):
    """Distinct experts of each token, the first ones hotter where skew > 0."""
    lg = torch.randn((T, E), generator=_gen(seed, 70), device=DEV)
    lg[:, : max(1, E // 8)] += skew
    return torch.topk(lg, k, dim=1).indices.to(torch.int32).contiguous()


def prepare(case, seed):
    c = dict(case)
    op = c["op"]
    if op in ("experts", "wgrad", "layer"):
        c["ids"] = _picks(c["T"], c["E"], c["k"], c["skew"], seed)
        c["most"] = int(torch.bincount(c["ids"].reshape(-1).long()).max())   # rows of the fullest expert
        P = c["T"] * c["k"]
    if op == "experts":
        c["X"] = _hidden(P if c["pairs"] else c["T"], c["K"], seed, 1)
        shape = (c["K"], c["N"]) if c["transposed"] else (c["N"], c["K"])
        c["W"] = _weights(c["E"], *shape, seed, 100)
    elif op == "wgrad":
        dy, x = (P, c["T"]) if c["side"] == "gate_up" else (c["T"], P)
        c["dY"] = _normal((dy, c["N"]), seed, 1)
        c["X"] = _hidden(x, c["K"], seed, 2)
        c["SX"] = None
        if c["codes"]:
            c["X"], c["SX"] = _quantize_rows(c["X"])
    elif op == "tn":
        c["A"] = _normal((c["M"], c["N"]), seed, 1)
        c["B"] = _hidden(c["M"], c["K"], seed, 2)
        c["SB"] = None
        if c["codes"]:
            c["B"], c["SB"] = _quantize_rows(c["B"])
    elif op == "swiglu":
        c["H1"] = _normal((c["R"], 2 * c["I"]), seed, 1, 2.0)
        c["SH"] = None
        if c["codes"]:
            c["H1"], c["SH"] = _quantize_rows(c["H1"])
        c["G"] = _normal((c["R"], c["I"]), seed, 2)
        c["w"] = torch.rand(c["R"], generator=_gen(seed, 3), device=DEV) if c["weights"] else None
    elif op == "linear":
        c["X"] = _hidden(c["M"], c["K"], seed, 1).requires_grad_()
        c["W"] = _normal((c["N"], c["K"]), seed, 2, 0.02).requires_grad_()
        c["dY"] = _normal((c["M"], c["N"]), seed, 3)
    else:
        T, E, H, I = c["T"], c["E"], c["H"], c["I"]
        c["X"] = _normal((T, H), seed, 1).requires_grad_()
        c["gate_up"] = _weights(E, 2 * I, H, seed, 100).requires_grad_()
        c["down"] = _weights(E, H, I, seed, 300).requires_grad_()
        w = torch.rand((T, c["k"]), generator=_gen(seed, 71), device=DEV) + 0.1
        c["w"] = (w / w.sum(1, keepdim=True)).to(BF16).requires_grad_()    # a bf16 model's router
        c["dOut"] = _normal((T, H), seed, 3)
    return c


# ------------------------------------------------------------------------------------------------ the plain forms --

def _pow2(e):
    """2^e for integers e, exactly, in fp32."""
    return ((e.long() + 1023) << 52).view(F64).to(F32)


def _quantize_rows(x):
    """e4m3 codes and e8m0 scales of bf16 rows, a scale per 128: 448 * 2^e = 0.875 * 2^(e + 9)."""
    x = x.float()
    M, K = x.shape
    nb = (K + 127) // 128
    v = torch.nn.functional.pad(x, (0, 128 * nb - K)).view(M, nb, 128)
    amax = v.abs().amax(2)
    m, p = torch.frexp(amax)
    e = torch.where(m <= 0.875, p - 9, p - 8).clamp(min=-127)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    q = (v * _pow2(-e)[:, :, None]).view(M, 128 * nb)[:, :K].contiguous().to(E4M3)
    s = torch.full((M, _cols(K)), 127, dtype=torch.uint8, device=x.device)
    s[:, :nb] = (e + 127).to(torch.uint8)
    return q, s.view(E8M0)


def _values(x, s):
    """fp32 values of bf16 rows (s None) or of codes with their scales."""
    if s is None:
        return x.float()
    K = x.shape[1]
    return x.float() * _pow2(s.view(torch.uint8).int() - 127).repeat_interleave(128, 1)[:, :K]


def _coded(x):
    return _values(*_quantize_rows(x))


def _fake_int4(w):
    """INT4 groups of 32: s = bf16(amax / 7), bf16(clamp(round(w / s)) s)."""
    v = w.float().view(*w.shape[:-1], -1, 32)
    s = (v.abs().amax(-1, keepdim=True) / 7).to(BF16).float()
    q = torch.where(s == 0, torch.zeros_like(v), torch.round(v / torch.where(s == 0, torch.ones_like(s), s)))
    return (q.clamp(-8, 7) * s).to(BF16).view(w.shape).float()


def _blocks_coded(w):
    """Values of a weight quantized in blocks of 128 x 128."""
    N, K = w.shape
    nn, nk = (N + 127) // 128, (K + 127) // 128
    v = torch.nn.functional.pad(w.float(), (0, 128 * nk - K, 0, 128 * nn - N)).view(nn, 128, nk, 128)
    amax = v.abs().amax((1, 3), keepdim=True)
    m, p = torch.frexp(amax)
    e = torch.where(m <= 0.875, p - 9, p - 8).clamp(min=-127)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    q = (v * _pow2(-e)).to(E4M3).float() * _pow2(e)
    return q.view(128 * nn, 128 * nk)[:N, :K].contiguous()


class _Rows:
    """Pairs grouped by expert: gather to [E, most] rows (zeros behind an expert's last one) and back."""

    def __init__(self, ids, E, most):
        flat = ids.reshape(-1).long()
        count = torch.bincount(flat, minlength=E)
        self.pairs, self.E, self.most = flat.numel(), E, most
        self.order = torch.argsort(flat, stable=True)
        self.expert = flat[self.order]
        self.place = torch.arange(self.pairs, device=ids.device) - (torch.cumsum(count, 0) - count)[self.expert]

    def gather(self, x):
        out = torch.zeros((self.E, self.most, x.shape[1]), dtype=x.dtype, device=x.device)
        out[self.expert, self.place] = x[self.order // (self.pairs // x.shape[0])]
        return out

    def back(self, y):
        out = torch.empty((self.pairs, y.shape[2]), dtype=y.dtype, device=y.device)
        out[self.order] = y[self.expert, self.place]
        return out

    def product(self, x, w):
        """Row f: x's row times w[e], w [E, K, N] contiguous."""
        return self.back(torch.bmm(self.gather(x), w))

    def outer(self, dy, x):
        return torch.bmm(self.gather(dy).transpose(1, 2).contiguous(), self.gather(x))


def _t(w):
    return w.transpose(-1, -2).contiguous()


def _swiglu_grads(h, G, w):
    g, u = h.chunk(2, -1)
    s = 1 / (1 + torch.exp(-g))
    a = g * s * u
    d = G if w is None else G * w[:, None]
    dh = torch.cat([d * u * s * (1 + g * (1 - s)), d * g * s], 1)
    return dh.to(BF16), (a if w is None else a * w[:, None]).to(BF16), (G * a).sum(1)


def _plain(c):
    op = c["op"]
    if op == "experts":
        W = c["W"].float()
        return _Rows(c["ids"], c["E"], c["most"]).product(c["X"].float(), W if c["transposed"] else _t(W)).to(BF16)
    if op == "wgrad":
        return _Rows(c["ids"], c["E"], c["most"]).outer(c["dY"].float(), _values(c["X"], c["SX"])).to(BF16)
    if op == "tn":
        return c["A"].float().t().matmul(_values(c["B"], c["SB"])).to(BF16)
    if op == "swiglu":
        dh, a, dw = _swiglu_grads(_values(c["H1"], c["SH"]), c["G"].float(), c["w"])
        return {"dH1": dh, "A": a, "dw": dw} if c["weights"] else {"dH1": dh, "A": a}
    if op == "linear":
        X, W, dY = c["X"].detach(), c["W"].detach(), c["dY"].float()
        Wf = _blocks_coded(W) if c["kind"] == "w8" else _fake_int4(W)
        xq = _coded(X)
        Y = (xq if c["kind"] == "w8" else X.float()).matmul(Wf.t()).to(BF16)
        dX = (_coded(dY) if c["kind"] == "w8" else dY).matmul(Wf).to(BF16)
        return {"Y": Y, "dX": dX, "dW": dY.t().matmul(xq).to(BF16)}
    with torch.no_grad():
        T, k = c["T"], c["k"]
        rows = _Rows(c["ids"], c["E"], c["most"])
        X, w = c["X"].detach(), c["w"].detach().float()
        Wu = _fake_int4(c["gate_up"]) if c["int4"] else c["gate_up"].detach().float()
        Wd = _fake_int4(c["down"]) if c["int4"] else c["down"].detach().float()
        h = rows.product(X.float(), _t(Wu)).to(BF16)
        g, u = h.float().chunk(2, 1)
        a = (g / (1 + torch.exp(-g)) * u).to(BF16)
        h2 = rows.product(a.float(), _t(Wd)).to(BF16)
        out = (h2.float().view(T, k, -1) * w[:, :, None]).sum(1).to(BF16)
        dO = c["dOut"].float()
        G = rows.product(dO, Wd).to(BF16)
        dh, aw, dw = _swiglu_grads(_coded(h) if c["checkpoint"] else h.float(), G.float(), w.reshape(-1))
        dXp = rows.product(dh.float(), Wu).to(BF16)
        return {"out": out, "dX": dXp.float().view(T, k, -1).sum(1).to(BF16), "dw": dw.to(BF16).view(T, k),
                "dgate_up": rows.outer(dh.float(), _coded(X) if c["checkpoint"] else X.float()).to(BF16),
                "ddown": rows.outer(dO, aw.float()).to(BF16)}


# --------------------------------------------------------------------------------------------- the package's calls --

def _calls(c):
    import int4_weight_only_amd as w4
    from int4_weight_only_amd import moe, qat, w8
    op = c["op"]
    if op in ("experts", "wgrad"):
        T, k, E = c["T"], c["k"], c["E"]
        B = w4.w4_bf16_pick_block_size(T, k, E)
        plan = w4.moe_align_block_size(c["ids"], E, B)
        if op == "experts":
            return w4.w4_bf16_moe_gemm(c["X"], c["W"], *plan, T, k, B, 1 if c["pairs"] else k,
                                       transposed=c["transposed"])
        dy_div, x_div = (1, k) if c["side"] == "gate_up" else (k, 1)
        return w4.w4_bf16_moe_wgrad(c["dY"], c["X"], *plan, E, T, k, B, dy_div, x_div, SX=c["SX"])
    if op == "tn":
        return w4.w4_bf16_gemm_tn(c["A"], c["B"], SB=c["SB"])
    if op == "swiglu":
        dh, a, dw = w4.w4_silu_mul_bwd(c["H1"], c["G"], weights=c["w"], SH=c["SH"])
        return {"dH1": dh, "A": a, "dw": dw} if c["weights"] else {"dH1": dh, "A": a}
    if op == "linear":
        layer = w8.w8_linear if c["kind"] == "w8" else qat.qat_linear
        Y = layer(c["X"], c["W"], checkpoint=True)
        dX, dW = torch.autograd.grad(Y, (c["X"], c["W"]), c["dY"])
        return {"Y": Y.detach(), "dX": dX, "dW": dW}
    inputs = (c["X"], c["w"], c["gate_up"], c["down"])
    out = moe.moe_train(c["X"], c["ids"], c["w"].float(), c["gate_up"], c["down"], int4=c["int4"],
                        checkpoint=c["checkpoint"])
    dX, dw, du, dd = torch.autograd.grad(out, inputs, c["dOut"])
    return {"out": out.detach(), "dX": dX, "dw": dw, "dgate_up": du, "ddown": dd}


def run(state):
    return _calls(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------ the definitions, 64 bits --

def _e4m3_64(v):
    """v rounded to the e4m3 grid (steps of 2^-9 below 2^-6, of an eighth of the binade above), ties to even."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))).round() - 3)
    return torch.round(v / step) * step


def _coded_64(x, tall=1):
    """Values of x quantized with one power of two per block of ``tall`` x 128, found by search from below."""
    R, C = x.shape
    x = x.double()
    amax = torch.nn.functional.max_pool2d(
        torch.nn.functional.pad(x.abs(), (0, -C % 128, 0, -R % tall))[None, None], (tall, 128))[0, 0]
    e = torch.floor(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax)))).round() - 9
    for _ in range(3):
        e = torch.where(amax > 448 * torch.exp2(e), e + 1, e)
    s = torch.exp2(torch.where(amax > 0, e.clamp(min=-127), torch.zeros_like(e)))
    s = s.repeat_interleave(tall, 0)[:R].repeat_interleave(128, 1)[:, :C]
    return _e4m3_64(x / s) * s


def _stored_64(x, s):
    if s is None:
        return x.double()
    scale = torch.exp2(s.view(torch.uint8).double() - 127)
    return x.float().double() * scale.repeat_interleave(128, 1)[:, : x.shape[1]]


def _int4_64(w):
    v = w.double().unflatten(-1, (-1, 32))
    s = (v.abs().amax(-1, keepdim=True) / 7).to(F32).to(BF16).double()
    q = torch.where(s > 0, torch.round(v / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(v))
    return (q.clamp(-8, 7) * s).to(BF16).double().flatten(-2)


def _each(ids, E):
    """(expert, its pairs in ascending order) for every expert."""
    flat = ids.reshape(-1)
    for e in range(E):
        yield e, torch.nonzero(flat == e)[:, 0]


def _rows_64(X, W, ids, transposed):
    """Expert by expert: X's row of every pair times W[e]^T, or W[e]."""
    P = ids.numel()
    out = torch.empty((P, W.shape[2] if transposed else W.shape[1]), dtype=F64, device=X.device)
    for e, f in _each(ids, W.shape[0]):
        w = W[e].double()
        out[f] = X[f // (P // X.shape[0])].double() @ (w if transposed else w.t())
    return out


def _outer_64(dY, X, ids, E):
    P = ids.numel()
    out = torch.zeros((E, dY.shape[1], X.shape[1]), dtype=F64, device=X.device)
    for e, f in _each(ids, E):
        out[e] = dY[f // (P // dY.shape[0])].double().t() @ X[f // (P // X.shape[0])]
    return out


def _swiglu_64(h, G, w):
    """By differentiating the definition."""
    h = h.double().requires_grad_()
    g, u = h.chunk(2, 1)
    a = g * torch.sigmoid(g) * u
    d = G.double() * (w.double()[:, None] if w is not None else 1)
    dh = torch.autograd.grad(a, h, d)[0]
    a = a.detach()
    return dh, a * w.double()[:, None] if w is not None else a, (G.double() * a).sum(1)


def exact(case, seed):
    c = prepare(case, seed)
    op = c["op"]
    if op == "experts":
        return _rows_64(c["X"], c["W"], c["ids"], c["transposed"])
    if op == "wgrad":
        return _outer_64(c["dY"], _stored_64(c["X"], c["SX"]), c["ids"], c["E"])
    if op == "tn":
        return c["A"].double().t() @ _stored_64(c["B"], c["SB"])
    if op == "swiglu":
        dh, a, dw = _swiglu_64(_stored_64(c["H1"], c["SH"]), c["G"], c["w"])
        return {"dH1": dh, "A": a, "dw": dw} if c["weights"] else {"dH1": dh, "A": a}
    if op == "linear":
        X, W, dY = c["X"].detach(), c["W"].detach(), c["dY"]
        xq = _coded_64(X)
        if c["kind"] == "w8":
            Wf = _coded_64(W, 128)
            return {"Y": xq @ Wf.t(), "dX": _coded_64(dY) @ Wf, "dW": dY.double().t() @ xq}
        Wf = _int4_64(W)
        return {"Y": X.double() @ Wf.t(), "dX": dY.double() @ Wf, "dW": dY.double().t() @ xq}
    T, k, E, ids = c["T"], c["k"], c["E"], c["ids"]
    X, w, dO = c["X"].detach(), c["w"].detach(), c["dOut"]
    Wu, Wd = c["gate_up"].detach(), c["down"].detach()
    if c["int4"]:
        Wu, Wd = _int4_64(Wu).to(BF16), _int4_64(Wd).to(BF16)
    h = _rows_64(X, Wu, ids, False).to(BF16)
    g, u = h.double().chunk(2, 1)
    a = (g * torch.sigmoid(g) * u).to(BF16)
    h2 = _rows_64(a, Wd, ids, False).to(BF16).double()
    out = (h2.view(T, k, -1) * w.double()[:, :, None]).sum(1)
    G = _rows_64(dO, Wd, ids, True).to(BF16)
    dh, aw, dw = _swiglu_64(_coded_64(h) if c["checkpoint"] else h, G, w.reshape(-1))
    dh, aw = dh.to(BF16), aw.to(BF16).double()
    return {"out": out, "dX": _rows_64(dh, Wu, ids, True).to(BF16).double().view(T, k, -1).sum(1),
            "dw": dw.view(T, k),
            "dgate_up": _outer_64(dh, _coded_64(X) if c["checkpoint"] else X.double(), ids, E),
            "ddown": _outer_64(dO, aw, ids, E)}
