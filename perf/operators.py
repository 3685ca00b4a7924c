"""The FP8 operators and the scored router, as cases to measure.

``run`` computes a case in its plain form (elementary torch operations in 32 bits, 64 where values lie next to a
border), or, where ``own`` is true, by the calls of this repository's package.  ``exact`` gives the same outputs from
the definitions in 64 bits.

Definitions (codes are e4m3, scales e8m0, that is powers of two; SC(K) = 4 ceil(K / 512) scale bytes a row):
  quantize   per block of 128: e = smallest integer >= -127 with amax <= 448 * 2^e (0 for a block of zeros),
             code = e4m3(x * 2^-e)
  product    Y[m, n] = bf16(sum_k X8[m, k] 2^SX[m, k/128] W8[n, k] 2^SW[n/128, k/128])
  router     s = sigmoid or softmax of the logits, c = s + bias; the best groups by the sum of their largest c, the k
             largest c in them (ties to the lowest index), weights from s
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


# ----------------------------------------------------------------------------------------------------- the cases --

def listed():
    return [
        # a decode step's router: 16 sequences, group-limited softmax, weights as they are
        dict(name="route_serve", op="route", T=16, E=128, k=8, sigmoid=False, bias=False, groups=8, topk_groups=4,
             group_top=1, renorm=False, scale=4.0, train=False),
        # a training batch's router with its gradient: sigmoid scores, balance bias, groups by their best two
        dict(name="route_train", op="route", T=16384, E=384, k=8, sigmoid=True, bias=True, groups=8, topk_groups=4,
             group_top=2, renorm=True, scale=2.5, train=True),
        # activations of a decode step, quantized before a projection
        dict(name="quantize_rows", op="rows", M=32, K=4096),
        # a weight at its update, codes in both directions (forward and input gradient)
        dict(name="quantize_weight", op="blocks", N=14336, K=4096, transposed=True),
        # between the two expert products: 256 tokens x 8 picks
        dict(name="silu_decode", op="silu", R=2048, I=2048),
        # the same in prefill, odd rows and a last block of 80
        dict(name="silu_prefill", op="silu", R=32775, I=2000),
        # one token against a projection
        dict(name="gemm_token", op="gemm", M=1, N=12288, K=4096),
        # a small batch, nothing a multiple of a tile
        dict(name="gemm_ragged", op="gemm", M=333, N=4101, K=7184),
        # a prefill's projection
        dict(name="gemm_prefill", op="gemm", M=4096, N=14336, K=4096),
        # a training step of a linear layer: output, both gradients
        dict(name="linear_train", op="linear", M=2050, N=4096, K=5120),
        # the experts' first product of a decode step, bound by reading the weights
        dict(name="experts_decode", op="experts", T=256, E=128, k=8, N=4096, K=4096, skew=0.0),
        # a whole routed layer in prefill, some experts hotter than others
        dict(name="layer_prefill", op="layer", T=2048, E=32, k=8, H=4096, I=2048, skew=1.0),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["route", "rows", "blocks", "silu", "gemm", "gemm", "linear", "experts", "layer"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * rng.randint(max(2, 16 // groups), 384 // groups)
        topk_groups = rng.randint((groups + 1) // 2, groups)
        k = rng.randint(1, min(8, topk_groups * (E // groups)))
        return dict(op=op, T=_log(rng, 1, 16384), E=E, k=k, sigmoid=rng.random() < 0.5, bias=rng.random() < 0.5,
                    groups=groups, topk_groups=topk_groups, group_top=rng.choice([1, 2]), renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), train=rng.random() < 0.5)
    if op == "rows":
        return dict(op=op, M=_log(rng, 1, 8192), K=_log(rng, 128, 8192, 16))
    if op == "blocks":
        return dict(op=op, N=_log(rng, 128, 14336, 16), K=_log(rng, 128, 4096, 16), transposed=rng.random() < 0.5)
    if op == "silu":
        return dict(op=op, R=_log(rng, 1, 32768), I=_log(rng, 64, 2048, 16))
    if op == "gemm":
        return dict(op=op, M=_log(rng, 1, 4096), N=_log(rng, 64, 14336), K=_log(rng, 128, 4096, 16))
    if op == "linear":
        return dict(op=op, M=_log(rng, 1, 2048), N=_log(rng, 64, 4096, 16), K=_log(rng, 128, 4096, 16))
    E = rng.choice([4, 8, 16, 32, 64])
    k = rng.randint(1, min(8, E))
    if op == "experts":
        return dict(op=op, T=_log(rng, 1, 2048), E=E, k=k, N=_log(rng, 64, 4096), K=_log(rng, 128, 4096, 16),
                    skew=rng.choice([0.0, 1.0]))
    return dict(op=op, T=_log(rng, 1, 1024), E=min(E, 32), k=min(k, 8), H=_log(rng, 128, 4096, 16),
                I=_log(rng, 64, 2048, 16), skew=rng.choice([0.0, 1.0]))


def _cols(K):
    return 4 * ((K + 511) // 512)


def _blocks(n):
    return (n + 127) // 128


def _used(c):
    """Experts that draw tokens: no more than there are pairs."""
    return min(c["E"], c["T"] * c["k"])


def work(case):
    c = case
    if c["op"] == "route":
        te, tk = c["T"] * c["E"], c["T"] * c["k"]
        b, f = 4 * te + 8 * tk, 8 * te
        if c["train"]:
            b, f = b + 8 * te + 12 * tk, f + 8 * te
    elif c["op"] == "rows":
        b, f = c["M"] * (3 * c["K"] + _cols(c["K"])), 3 * c["M"] * c["K"]
    elif c["op"] == "blocks":
        b = c["N"] * c["K"] * (4 if c["transposed"] else 3) + _blocks(c["N"]) * _cols(c["K"])
        f = 3 * c["N"] * c["K"]
    elif c["op"] == "silu":
        b, f = c["R"] * (5 * c["I"] + _cols(c["I"])), 10 * c["R"] * c["I"]
    elif c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        b = M * (K + _cols(K)) + N * K + _blocks(N) * _cols(K) + 2 * M * N
        f = 2 * M * N * K
    elif c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        b, f = 4 * M * K + 4 * N * K + 4 * M * N, 6 * M * N * K
    elif c["op"] == "experts":
        P, N, K = c["T"] * c["k"], c["N"], c["K"]
        b = c["T"] * (K + _cols(K)) + _used(c) * N * K + 2 * P * N
        f = 2 * P * N * K
    else:
        P, H, I = c["T"] * c["k"], c["H"], c["I"]
        b = 4 * c["T"] * H + 4 * c["T"] * c["E"] + _used(c) * 3 * H * I
        f = 6 * P * H * I
    return {"bytes": b, "flops": f}


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
    """Block-quantized weights of E experts, N(0, 0.02)."""
    W8 = torch.empty((E, N, K), dtype=E4M3, device=DEV)
    SW = torch.empty((E, _blocks(N), _cols(K)), dtype=E8M0, device=DEV)
    for e in range(E):
        W8[e], s = _quantize_blocks(_normal((N, K), seed, stream + e, 0.02))
        SW[e].view(torch.uint8).copy_(s.view(torch.uint8))
    return W8, SW


def _picks(T, E, k, skew, seed):
    """Distinct experts of each token, the first ones hotter where skew > 0."""
    lg = torch.randn((T, E), generator=_gen(seed, 70), device=DEV)
    lg[:, : max(1, E // 8)] += skew
    return torch.topk(lg, k, dim=1).indices.to(torch.int32).contiguous()


def prepare(case, seed):
    c = dict(case)
    op = c["op"]
    if op == "route":
        c["logits"] = torch.randn((c["T"], c["E"]), generator=_gen(seed, 1), device=DEV)
        b = torch.randn(c["E"], generator=_gen(seed, 2), device=DEV) * 0.05
        c["bias_t"] = b if c["bias"] else None
        c["dw"] = torch.randn((c["T"], c["k"]), generator=_gen(seed, 3), device=DEV)
    elif op == "rows":
        c["X"] = _hidden(c["M"], c["K"], seed, 1)
    elif op == "blocks":
        c["W"] = _normal((c["N"], c["K"]), seed, 1, 0.02)
    elif op == "silu":
        c["H1"] = _normal((c["R"], 2 * c["I"]), seed, 1)
    elif op == "gemm":
        c["X8"], c["SX"] = _quantize_rows(_hidden(c["M"], c["K"], seed, 1))
        c["W8"], c["SW"] = _quantize_blocks(_normal((c["N"], c["K"]), seed, 2, 0.02))
    elif op == "linear":
        c["X"] = _hidden(c["M"], c["K"], seed, 1).requires_grad_()
        c["W"] = _normal((c["N"], c["K"]), seed, 2, 0.02).requires_grad_()
        c["dY"] = _normal((c["M"], c["N"]), seed, 3)
    elif op == "experts":
        c["X8"], c["SX"] = _quantize_rows(_hidden(c["T"], c["K"], seed, 1))
        c["W8"], c["SW"] = _weights(c["E"], c["N"], c["K"], seed, 100)
        c["ids"] = _picks(c["T"], c["E"], c["k"], c["skew"], seed)
        c["most"] = int(torch.bincount(c["ids"].reshape(-1).long()).max())   # rows of the fullest expert
    else:
        T, E, k, H, I = c["T"], c["E"], c["k"], c["H"], c["I"]
        c["X"] = _normal((T, H), seed, 1)
        c["gate_up"] = _weights(E, 2 * I, H, seed, 100)
        c["down"] = _weights(E, H, I, seed, 300)
        lg = torch.randn((T, E), generator=_gen(seed, 70), device=DEV)
        lg[:, : max(1, E // 8)] += c["skew"]
        c["logits"] = lg
        c["bias_t"] = torch.randn(E, generator=_gen(seed, 71), device=DEV) * 0.05
        ids, _ = _route(lg, c["bias_t"], k, True, 1, 1, 1, True, 2.5)
        c["most"] = int(torch.bincount(ids.reshape(-1).long()).max())        # rows of the fullest expert
    return c


# ------------------------------------------------------------------------------------------------ the plain forms --

def _pow2(e):
    """2^e for integers e, exactly, in fp32."""
    return ((e.long() + 1023) << 52).view(F64).to(F32)


def _exponent(amax):
    """Smallest e >= -127 with amax <= 448 * 2^e; 0 for amax = 0.  448 * 2^e = 0.875 * 2^(e + 9)."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8).clamp(min=-127)
    return torch.where(amax == 0, torch.zeros_like(e), e)


def _scale_bytes(e, cols):
    """Exponents [R, blocks] as e8m0 [R, cols], padding 1.0."""
    s = torch.full((e.shape[0], cols), 127, dtype=torch.uint8, device=e.device)
    s[:, : e.shape[1]] = (e + 127).to(torch.uint8)
    return s.view(E8M0)


def _pad(x, rows, cols):
    return torch.nn.functional.pad(x, (0, cols - x.shape[1], 0, rows - x.shape[0]))


def _quantize_rows(x):
    x = x.float()
    M, K = x.shape
    nb = _blocks(K)
    v = _pad(x, M, 128 * nb).view(M, nb, 128)
    e = _exponent(v.abs().amax(2))
    q = (v * _pow2(-e)[:, :, None]).view(M, 128 * nb)[:, :K].contiguous().to(E4M3)
    return q, _scale_bytes(e, _cols(K))


def _block_codes(w):
    N, K = w.shape
    nn, nk = _blocks(N), _blocks(K)
    v = _pad(w.float(), 128 * nn, 128 * nk).view(nn, 128, nk, 128)
    e = _exponent(v.abs().amax((1, 3)))
    q = (v * _pow2(-e)[:, None, :, None]).view(128 * nn, 128 * nk)[:N, :K]
    return q, e


def _quantize_blocks(w):
    q, e = _block_codes(w)
    return q.contiguous().to(E4M3), _scale_bytes(e, _cols(w.shape[1]))


def _values(s, blocks):
    """Scale bytes -> fp32 values of the first ``blocks`` columns."""
    return _pow2(s.view(torch.uint8)[..., :blocks].int() - 127)


def _rows_f32(X8, SX):
    K = X8.shape[1]
    s = _values(SX, _blocks(K))
    return X8.float() * s.repeat_interleave(128, 1)[:, :K]


def _blocks_f32(W8, SW):
    N, K = W8.shape[-2:]
    s = _values(SW, _blocks(K))
    s = s.repeat_interleave(128, -1)[..., :K].repeat_interleave(128, -2)[..., :N, :]
    return W8.float() * s


def _silu_mul(h):
    g, u = h.float().chunk(2, -1)
    return g / (1 + torch.exp(-g)) * u


def _score(x, sigmoid):
    x = x.double()
    if sigmoid:
        return 1 / (1 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _route(logits, bias, k, sigmoid, groups, topk_groups, group_top, renorm, scale):
    T, E = logits.shape
    s = _score(logits, sigmoid)
    c = s + bias.double() if bias is not None else s
    if groups > 1:
        per = c.view(T, groups, E // groups)
        value = per.topk(min(group_top, E // groups), 2).values.sum(2)
        best = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :topk_groups]
        keep = torch.zeros_like(value, dtype=torch.bool).scatter_(1, best, True)
        c = torch.where(keep[:, :, None], per, torch.full_like(per, -math.inf)).view(T, E)
    ids = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, ids)
    if renorm:
        w = w / w.sum(1, keepdim=True)
    return ids.to(torch.int32), (scale * w).float()


def _route_grad(logits, ids, dw, sigmoid, renorm, scale):
    s = _score(logits, sigmoid)
    ids, g = ids.long(), scale * dw.double()
    p = s.gather(1, ids)
    out = torch.zeros_like(s)
    if renorm:
        w = p / p.sum(1, keepdim=True)
        d = w * (g - (g * w).sum(1, keepdim=True))
        d = d * (1 - p) if sigmoid else d
    elif sigmoid:
        d = g * p * (1 - p)
    else:
        d = g * p
        out = -s * d.sum(1, keepdim=True)
    return out.scatter_add(1, ids, d).float()


def _grouped(X, W, ids, most):
    """Row f = t k + j of the result: X's row f (or token t's) times W[ids[t, j]]^T, all in X's type.  Rows are
    gathered by expert into [E, most], multiplied, and put back."""
    E, P = W.shape[0], ids.numel()
    flat = ids.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    expert = flat[order]
    start = torch.cumsum(torch.bincount(flat, minlength=E), 0) - torch.bincount(flat, minlength=E)
    place = torch.arange(P, device=X.device) - start[expert]
    rows = X[order // (P // X.shape[0])]
    padded = torch.zeros((E, most, X.shape[1]), dtype=X.dtype, device=X.device)
    padded[expert, place] = rows
    y = torch.bmm(padded, W.transpose(1, 2).contiguous())
    out = torch.empty((P, W.shape[1]), dtype=X.dtype, device=X.device)
    out[order] = y[expert, place]
    return out


def _plain(c):
    op = c["op"]
    if op == "route":
        ids, w = _route(c["logits"], c["bias_t"], c["k"], c["sigmoid"], c["groups"], c["topk_groups"],
                        c["group_top"], c["renorm"], c["scale"])
        if not c["train"]:
            return {"ids": ids, "weights": w}
        return {"ids": ids, "weights": w,
                "dlogits": _route_grad(c["logits"], ids, c["dw"], c["sigmoid"], c["renorm"], c["scale"])}
    if op == "rows":
        q, s = _quantize_rows(c["X"])
        return {"codes": q, "scales": s.view(torch.uint8)}
    if op == "blocks":
        q, e = _block_codes(c["W"])
        N, K = q.shape
        got = {"codes": q.contiguous().to(E4M3), "scales": _scale_bytes(e, _cols(K)).view(torch.uint8)}
        if c["transposed"]:
            got["codes_t"] = q.t().contiguous().to(E4M3)
            got["scales_t"] = _scale_bytes(e.t(), _cols(N)).view(torch.uint8)
        return got
    if op == "silu":
        q, s = _quantize_rows(_silu_mul(c["H1"]))
        return {"codes": q, "scales": s}
    if op == "gemm":
        return _rows_f32(c["X8"], c["SX"]).matmul(_blocks_f32(c["W8"], c["SW"]).t()).to(BF16)
    if op == "linear":
        X, W, dY = c["X"].detach(), c["W"].detach(), c["dY"]
        Wf = _blocks_f32(*_quantize_blocks(W))
        return {"Y": _rows_f32(*_quantize_rows(X)).matmul(Wf.t()).to(BF16),
                "dX": _rows_f32(*_quantize_rows(dY)).matmul(Wf).to(BF16),
                "dW": dY.float().t().matmul(X.float()).to(BF16)}
    if op == "experts":
        return _grouped(_rows_f32(c["X8"], c["SX"]), _blocks_f32(c["W8"], c["SW"]), c["ids"], c["most"]).to(BF16)
    ids, w = _route(c["logits"], c["bias_t"], c["k"], True, 1, 1, 1, True, 2.5)
    h1 = _grouped(_rows_f32(*_quantize_rows(c["X"])), _blocks_f32(*c["gate_up"]), ids, c["most"]).to(BF16)
    h2 = _grouped(_rows_f32(*_quantize_rows(_silu_mul(h1))), _blocks_f32(*c["down"]), ids, c["most"]).to(BF16)
    out = (h2.float().view(c["T"], c["k"], -1) * w[:, :, None]).sum(1).to(BF16)
    return {"out": out, "ids": ids, "weights": w}


# --------------------------------------------------------------------------------------------- the package's calls --

def _calls(c):
    import int4_weight_only_amd as w4
    from int4_weight_only_amd import moe, w8
    op = c["op"]
    if op == "route":
        how = dict(sigmoid=c["sigmoid"], renorm=c["renorm"], scale=c["scale"])
        ids, w = w4.w4_moe_route_scored(c["logits"], c["k"], bias=c["bias_t"], groups=c["groups"],
                                        topk_groups=c["topk_groups"], group_top=c["group_top"], **how)
        if not c["train"]:
            return {"ids": ids, "weights": w}
        return {"ids": ids, "weights": w,
                "dlogits": w4.w4_moe_route_scored_bwd(c["logits"], ids, w, c["dw"], **how)}
    if op == "rows":
        q, s = w4.w8_quantize_rows(c["X"])
        return {"codes": q, "scales": s.view(torch.uint8)}
    if op == "blocks":
        q, s, qt, st = w4.w8_quantize_blocks(c["W"], transposed=c["transposed"])
        got = {"codes": q, "scales": s.view(torch.uint8)}
        if c["transposed"]:
            got["codes_t"], got["scales_t"] = qt, st.view(torch.uint8)
        return got
    if op == "silu":
        q, s = w4.w8_silu_mul_quantize(c["H1"])
        return {"codes": q, "scales": s}
    if op == "gemm":
        return w4.w8a8_gemm(c["X8"], c["SX"], c["W8"], c["SW"])
    if op == "linear":
        Y = w8.w8_linear(c["X"], c["W"])
        dX, dW = torch.autograd.grad(Y, (c["X"], c["W"]), c["dY"])
        return {"Y": Y, "dX": dX, "dW": dW}
    if op == "experts":
        B = w4.w8_pick_block_size(c["T"], c["k"], c["E"])
        plan = w4.moe_align_block_size(c["ids"], c["E"], B)
        return w4.w8a8_moe_gemm(c["X8"], c["SX"], c["W8"], c["SW"], *plan, c["T"], c["k"], B, c["k"])
    out, ids, w, _ = moe.moe_layer_w8(c["X"], c["logits"], c["k"], moe.ExpertWeightsW8(*c["gate_up"]),
                                      moe.ExpertWeightsW8(*c["down"]), sigmoid=True, bias=c["bias_t"], scale=2.5)
    return {"out": out, "ids": ids, "weights": w}


def run(state):
    return _calls(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------ the definitions, 64 bits --

def _e4m3_64(v):
    """v rounded to the e4m3 grid (steps of 2^-9 below 2^-6, of an eighth of the binade above), ties to even."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))).round() - 3)
    return torch.round(v / step) * step


def _shift_64(amax):
    """The exponent of a block's scale, by search from below."""
    e = torch.floor(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax)))).round() - 9
    for _ in range(3):
        e = torch.where(amax > 448 * torch.exp2(e), e + 1, e)
    return torch.where(amax > 0, e.clamp(min=-127), torch.zeros_like(e))


def _quant_64(x, tall):
    """(codes, scales spread over x's shape, exponents of the blocks) of blocks of ``tall`` x 128."""
    R, C = x.shape
    x = x.double()
    amax = torch.nn.functional.max_pool2d(
        torch.nn.functional.pad(x.abs(), (0, -C % 128, 0, -R % tall))[None, None], (tall, 128))[0, 0]
    e = _shift_64(amax)
    s = torch.exp2(e).repeat_interleave(tall, 0)[:R].repeat_interleave(128, 1)[:, :C]
    return _e4m3_64(x / s), s, e


def _stored_64(codes, scales, tall):
    R, C = codes.shape[-2:]
    s = torch.exp2(scales.view(torch.uint8).double() - 127)
    s = s.repeat_interleave(tall, -2)[..., :R, :].repeat_interleave(128, -1)[..., :C]
    return codes.float().double() * s


def _scores_64(x, sigmoid):
    x = x.double()
    return torch.sigmoid(x) if sigmoid else torch.softmax(x, 1)


def _first_64(v, k):
    """Indices of the k largest values of each row, ties to the lowest index."""
    v = v.cpu().numpy()
    return np.argsort(-v, axis=1, kind="stable")[:, :k]


def _picks_64(logits, bias, k, sigmoid, groups, topk_groups, group_top):
    c = _scores_64(logits, sigmoid)
    c = c if bias is None else c + bias.double()
    per = c.view(c.shape[0], groups, -1)
    best = _first_64(per.sort(dim=2, descending=True).values[:, :, :group_top].sum(2), topk_groups)
    out = torch.ones(per.shape[:2], dtype=torch.bool)
    out[torch.arange(c.shape[0])[:, None], torch.from_numpy(best)] = False
    c = c.masked_fill(out.to(c.device).repeat_interleave(per.shape[2], 1), -math.inf)
    return torch.from_numpy(_first_64(c, k)).to(c.device)


def _weights_64(logits, ids, sigmoid, renorm, scale):
    s = _scores_64(logits, sigmoid)
    w = torch.take_along_dim(s, ids.long(), 1)
    return scale * (w / w.sum(1, keepdim=True) if renorm else w)


def _experts_64(X, W8, SW, ids):
    """Expert by expert, X's rows as _grouped takes them."""
    P = ids.numel()
    flat = ids.reshape(-1)
    out = torch.empty((P, W8.shape[1]), dtype=F64, device=X.device)
    for e in range(W8.shape[0]):
        f = torch.nonzero(flat == e)[:, 0]
        out[f] = X[f // (P // X.shape[0])] @ _stored_64(W8[e], SW[e], 128).t()
    return out


def exact(case, seed):
    c = prepare(case, seed)
    op = c["op"]
    if op == "route":
        ids = _picks_64(c["logits"], c["bias_t"], c["k"], c["sigmoid"], c["groups"], c["topk_groups"],
                        c["group_top"])
        x = c["logits"].double().requires_grad_()
        w = _weights_64(x, ids, c["sigmoid"], c["renorm"], c["scale"])
        got = {"ids": None, "weights": w.detach()}
        if c["train"]:
            got["dlogits"] = torch.autograd.grad(w, x, c["dw"].double())[0]
        return got
    if op == "rows":
        return {"codes": _quant_64(c["X"], 1)[0], "scales": None}
    if op == "blocks":
        q, _, _ = _quant_64(c["W"], 128)
        return {"codes": q, "scales": None, "codes_t": q.t().contiguous() if c["transposed"] else None,
                "scales_t": None}
    if op == "silu":
        g, u = c["H1"].double().chunk(2, 1)
        q, _, e = _quant_64(g * torch.sigmoid(g) * u, 1)
        s = torch.ones((c["R"], _cols(c["I"])), dtype=F64, device=q.device)
        s[:, : e.shape[1]] = torch.exp2(e)
        return {"codes": q, "scales": s}
    if op == "gemm":
        return _stored_64(c["X8"], c["SX"], 1) @ _stored_64(c["W8"], c["SW"], 128).t()
    if op == "linear":
        X, W, dY = c["X"].detach(), c["W"].detach(), c["dY"]
        Wq, Ws, _ = _quant_64(W, 128)
        Xq, Xs, _ = _quant_64(X, 1)
        Dq, Ds, _ = _quant_64(dY, 1)
        return {"Y": (Xq * Xs) @ (Wq * Ws).t(), "dX": (Dq * Ds) @ (Wq * Ws), "dW": dY.double().t() @ X.double()}
    if op == "experts":
        return _experts_64(_stored_64(c["X8"], c["SX"], 1), c["W8"], c["SW"], c["ids"])
    ids = _picks_64(c["logits"], c["bias_t"], c["k"], True, 1, 1, 1)
    w = _weights_64(c["logits"], ids, True, True, 2.5)
    q, s, _ = _quant_64(c["X"], 1)
    g, u = _experts_64(q * s, *c["gate_up"], ids).to(BF16).double().chunk(2, 1)
    q, s, _ = _quant_64(g * torch.sigmoid(g) * u, 1)
    h2 = _experts_64(q * s, *c["down"], ids).to(BF16).double()
    return {"out": (h2.view(c["T"], c["k"], -1) * w[:, :, None]).sum(1), "ids": None, "weights": w}
