"""Every kernel of the grouped and dense bf16 products, on small whole numbers: each sum is exact
in fp32 in any order (below 2^24), so that the result is the exact one rounded once to bf16 and is
compared bit for bit.  Few rows of one operand are not zero where a sum is long: results then
stay below 2^8, where bf16 holds every whole number, and a row lost or read elsewhere shows.
"""

import numpy as np
import pytest
import torch

import int4_weight_only_amd as w4
import train_tiles as tt
from gpu_util import CANARY, canary_bf16, dev, say, up

pytestmark = pytest.mark.gpu


def whole(shape, seed):
    """-1, 0 and 1 at random, bf16 on the GPU."""
    g = torch.Generator(device=dev()).manual_seed(seed)
    return torch.randint(-1, 2, shape, generator=g, device=dev(), dtype=torch.int8).to(torch.bfloat16)


def at(rows, t):
    """``t`` with zeros in all rows but ``rows``."""
    z = torch.zeros_like(t)
    z[rows] = t[rows]
    return z


def rounded(x):
    """fp64 whole numbers as bf16 (exact in fp32 on the way)."""
    assert float(x.abs().max()) < 1 << 24
    return x.float().to(torch.bfloat16)


def skewed(T, k, E, seed):
    """ids [T, k] with half of the pairs at one expert, one expert without any and a few pairs
    outside; every pair a draw of its own (the same expert twice in a token)."""
    r = np.random.default_rng(seed)
    live = [e for e in range(E) if e != 1] if E > 2 else list(range(E))
    ids = r.choice(live, (T, k))
    ids[r.random((T, k)) < 0.4] = live[-1]
    flat = ids.reshape(-1)
    if flat.size > 8:
        flat[r.permutation(flat.size)[:3]] = (-1, E, E + 5)
    return ids.astype(np.int32)


@pytest.mark.parametrize("T,k,E,N,K,B,tile,parts", tt.ROWS)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("per_pair", [False, True])
def test_rows(T, k, E, N, K, B, tile, parts, transposed, per_pair):
    say(f"rows T={T} k={k} E={E} N={N} K={K} B={B} tile={tile} parts={parts} transposed={transposed} per_pair={per_pair}")
    ids = skewed(T, k, E, N)
    div = 1 if per_pair else k
    X, W = whole((T * k // div, K), 1), whole((E, K, N) if transposed else (E, N, K), 2)
    out = canary_bf16((T * k, N))
    w4.w4_bf16_moe_gemm(X, W, *w4.moe_align_block_size(up(ids), E, B), T, k, B, div, transposed=transposed, out=out)
    flat = up(ids).reshape(-1)
    want = canary_bf16((T * k, N))
    for e in range(E):
        f = torch.nonzero(flat == e)[:, 0]
        if f.numel():
            we = W[e].double()
            want[f] = rounded(X[f // div].double() @ (we if transposed else we.t().contiguous()))
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))


def grouped_sums(ids, E, dY, X, dd, dx, rows=None):
    """dW of whole numbers; ``rows``: the pairs that are not zero in one of the operands."""
    flat = ids.reshape(-1).long()
    out = torch.zeros((E, dY.shape[1], X.shape[1]), dtype=torch.bfloat16, device=dev())
    for e in range(E):
        f = torch.nonzero(flat == e)[:, 0] if rows is None else rows[flat[rows] == e]
        if f.numel():
            out[e] = rounded(dY[f // dd].double().t().contiguous() @ X[f // dx].double())
    return out


@pytest.mark.parametrize("T,k,E,N,K,tile,parts", tt.SUMS)
@pytest.mark.parametrize("side", ["gate_up", "down"])
@pytest.mark.parametrize("codes", [False, True])
def test_sums(T, k, E, N, K, tile, parts, side, codes):
    say(f"sums T={T} k={k} E={E} N={N} K={K} tile={tile} parts={parts} {side} codes={codes}")
    B = 64 if T > 100000 else w4.w4_bf16_pick_block_size(T, k, E)
    ids = skewed(T, k, E, N)
    dd, dx = (1, k) if side == "gate_up" else (k, 1)
    dY, X, SX = whole((T * k // dd, N), 1), whole((T * k // dx, K), 2), None
    rows = None
    if T > 100000:                                    # k = 1: a pair is a row
        rows = torch.arange(0, T, 701, device=dev())
        dY = at(rows, dY)
    want = grouped_sums(up(ids), E, dY, X, dd, dx, rows)
    if codes:
        X, SX = w4.w8_quantize_rows(X)
    out = canary_bf16((E, N, K))
    w4.w4_bf16_moe_wgrad(dY, X, *w4.moe_align_block_size(up(ids), E, B), E, T, k, B, dd, dx, SX=SX, out=out)
    assert torch.equal(out, want)


@pytest.mark.parametrize("M,N,K,tile,parts", tt.DENSE)
@pytest.mark.parametrize("codes", [False, True])
def test_dense(M, N, K, tile, parts, codes):
    say(f"dense M={M} N={N} K={K} tile={tile} parts={parts} codes={codes}")
    A, B, SB = whole((M, N), 1), whole((M, K), 2), None
    want = rounded(A.double().t().contiguous() @ B.double())
    if codes:
        B, SB = w4.w8_quantize_rows(B)
    assert torch.equal(w4.w4_bf16_gemm_tn(A, B, SB=SB), want)


# ------------------------------------------------------------------- 2 GiB and more --

def marked(T, cols):
    """Rows at both ends, around 2^30, 2^31 and 2^32 of one and two bytes, and between."""
    rows = {*range(70), *range(T - 100, T), *range(0, T, 1009)}
    for where in (1 << 29, 1 << 30, 1 << 31):
        rows |= {r for r in range(where // cols - 20, where // cols + 20) if 0 <= r < T}
    return torch.tensor(sorted(rows), device=dev())


@pytest.mark.parametrize("T,N,K,B,tile", tt.WIDE_ROWS)
@pytest.mark.parametrize("transposed", [False, True])
def test_wide_rows(T, N, K, B, tile, transposed):
    say(f"wide rows T={T} N={N} K={K} B={B} tile={tile} transposed={transposed}")
    E = 2
    X, W = whole((T, K), 1), whole((E, K, N) if transposed else (E, N, K), 2)
    ids = torch.randint(0, E, (T, 1), generator=torch.Generator().manual_seed(3), dtype=torch.int32).to(dev())
    Y = w4.w4_bf16_moe_gemm(X, W, *w4.moe_align_block_size(ids, E, B), T, 1, B, 1, transposed=transposed)
    w = [(W[e] if transposed else W[e].t()).float().contiguous() for e in range(E)]
    for first in range(0, T, 1 << 14):
        x, one = X[first:first + (1 << 14)].float(), ids[first:first + (1 << 14)] == 1
        want = torch.where(one, x @ w[1], x @ w[0])
        assert torch.equal(Y[first:first + (1 << 14)], rounded(want)), first


@pytest.mark.parametrize("T,N,K,transposed,tile", tt.WIDE_WEIGHTS)
def test_wide_weights(T, N, K, transposed, tile):
    say(f"wide weights T={T} N={N} K={K} transposed={transposed}")
    cols = marked(K, N if transposed else 1)[::2]     # of X: rows of W where it lies across
    X = torch.zeros((T, K), dtype=torch.bfloat16, device=dev())
    X[:, cols] = whole((T, cols.numel()), 1)
    W = whole((1, K, N) if transposed else (1, N, K), 2)
    ids = torch.zeros((T, 1), dtype=torch.int32, device=dev())
    Y = w4.w4_bf16_moe_gemm(X, W, *w4.moe_align_block_size(ids, 1, 64), T, 1, 64, 1, transposed=transposed)
    w = W[0][cols].double() if transposed else W[0][:, cols].double().t().contiguous()
    assert torch.equal(Y, rounded(X[:, cols].double() @ w))


@pytest.mark.parametrize("T,E,N,K,codes,tile", tt.WIDE_SUMS)
def test_wide_sums(T, E, N, K, codes, tile):
    say(f"wide sums T={T} E={E} N={N} K={K} codes={codes} tile={tile}")
    rows = marked(T, max(N, K))
    A, B, SB = whole((T, N), 1), whole((T, K), 2), None
    if N < K:                                         # the narrow operand holds the zeros
        A = at(rows, A)
    else:
        B = at(rows, B)
    ids = torch.randint(0, E, (T, 1), generator=torch.Generator().manual_seed(3), dtype=torch.int32).to(dev())
    want = grouped_sums(ids, E, A, B, 1, 1, rows)
    if codes:
        B, SB = w4.w8_quantize_rows(B)
    plan = w4.moe_align_block_size(ids, E, 256)
    assert torch.equal(w4.w4_bf16_moe_wgrad(A, B, *plan, E, T, 1, 256, 1, 1, SX=SB), want)
    if E == 1:
        assert torch.equal(w4.w4_bf16_gemm_tn(A, B, SB=SB), want[0])
