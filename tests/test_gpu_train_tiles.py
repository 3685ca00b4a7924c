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
