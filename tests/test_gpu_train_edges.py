"""Training of the routed experts at the edges of what its calls allow.  Results that
must not depend on what was changed are compared bit for bit; a rounding to bf16 is half a
step, 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

import int4_weight_only_amd as w4
from gpu_util import dev, say, up
from int4_weight_only_amd import moe
from int4_weight_only_amd.qat import qat_linear
from int4_weight_only_amd.w8 import w8_linear
from oracle import train

pytestmark = pytest.mark.gpu

HALF, TINY = 2.0 ** -8, 2.0 ** -133


def normal(shape, seed, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * sigma).to(torch.bfloat16)


def spread(T, k, E):
    """ids [T, k]: token t's picks are t k, t k + 1, ... modulo E."""
    return ((np.arange(T * k) % E).reshape(T, k)).astype(np.int32)


# ------------------------------------------------------------------ gradients' addresses --

@pytest.mark.parametrize("layer", ["moe", "moe_int4", "moe_checkpoint", "w8", "w8_checkpoint", "int4", "int4_checkpoint"])
def test_gradient_at_any_address(layer):
    """The gradient that autograd hands to a layer may begin anywhere: here behind three values of
    a tensor that the output was joined with."""
    T, k, E, H, I = 20, 2, 4, 64, 32
    say(f"gradient at any address {layer}")
    if layer.startswith("moe"):
        ids, w = up(spread(T, k, E)), torch.full((T, k), 0.5, device=dev())
        base = [normal((T, H), 1).to(dev()), w, normal((E, 2 * I, H), 2, 0.2).to(dev()), normal((E, H, I), 3, 0.2).to(dev())]

        def f(X, w, gu, dn):
            return moe.moe_train(X, ids, w, gu, dn, int4="int4" in layer, checkpoint="checkpoint" in layer)
    else:
        base = [normal((T, H), 1).to(dev()), normal((64, H), 2).to(dev())]
        call = w8_linear if layer.startswith("w8") else qat_linear

        def f(X, W):
            return call(X, W, checkpoint="checkpoint" in layer)
    leaves = [t.clone().requires_grad_() for t in base]
    dO = normal((T * 64 + 3,), 4).to(dev())
    want = torch.autograd.grad(f(*leaves), leaves, dO[3:].clone().view(T, 64))
    joined = torch.cat([torch.zeros(3, device=dev(), dtype=torch.bfloat16), f(*leaves).reshape(-1)])
    for a, b in zip(want, torch.autograd.grad(joined, leaves, dO)):
        assert torch.equal(a, b)


# --------------------------------------------------------------------- refusals --

def test_moe_train_refuses_in_the_forward_what_the_backward_does_not_take():
    """Blocks of 16 are the INT4 product's, not the backward's: refused where a gradient is wanted,
    taken (and the same bits) where none is."""
    T, k, E, H, I = 20, 2, 4, 64, 32
    ids, w, X = up(spread(T, k, E)), torch.full((T, k), 0.5, device=dev()), normal((T, H), 1).to(dev())
    gu, dn = normal((E, 2 * I, H), 2, 0.2).to(dev()), normal((E, H, I), 3, 0.2).to(dev())
    out = moe.moe_train(X, ids, w, gu, dn, int4=True, B=16)
    assert torch.equal(out, moe.moe_train(X, ids, w, gu, dn, int4=True))
    for i in range(4):
        leaves = [t.clone().requires_grad_(n == i) for n, t in enumerate((X, w, gu, dn))]
        with pytest.raises(ValueError):
            moe.moe_train(leaves[0], ids, *leaves[1:], int4=True, B=16)
        with torch.no_grad():
            assert torch.equal(out, moe.moe_train(leaves[0], ids, *leaves[1:], int4=True, B=16))

# ----------------------------------------------------------------------- SwiGLU's range --

def test_silu_mul_bwd_large_factors():
    """Products whose factors pass fp32's range together while the result does not: the weight
    brings it back, the factor of u is above one, or the sigmoid lies below fp32's range."""
    top = 255 * 2.0 ** 120                            # the largest bf16
    rows = [(2.0 ** 30, 1.0, 2.0 ** 100, 2.0 ** -10),      # (g, u, dA, w)
            (2.0 ** 30, 1.0, 2.0 ** 110, 2.0 ** -20), (2.40625, top, 2.0 ** -10, 2.0 ** -4),
            (2.40625, -top, 2.0 ** -10, 2.0 ** -4), (1.5, 2.0 ** -20, top, 2.0 ** -3),
            (-84.0, 2.0 ** 127, 2.0 ** 60, 1.0), (-84.0, top, 2.0 ** 90, 2.0 ** -4),
            (-100.0, 2.0 ** 120, 2.0 ** 120, 2.0 ** -5), (-84.0, 2.0 ** -20, 2.0 ** 100, 0.5),
            (-84.0, 2.0 ** 100, 2.0 ** -20, 0.5), (-150.0, 2.0 ** 127, 2.0 ** 20, 0.5),
            (2.0 ** 70, 2.0 ** 70, 2.0 ** -60, 2.0 ** -20), (0.5, 2.0 ** -60, 2.0 ** 126, 0.25),
            (-80.0, 2.0 ** 10, 2.0 ** -20, 0.5)]
    I = 8
    v = np.array(rows)
    H1 = torch.from_numpy(np.concatenate([np.repeat(v[:, :1], I, 1), np.repeat(v[:, 1:2], I, 1)], 1)).to(torch.bfloat16)
    G = torch.from_numpy(np.repeat(v[:, 2:3], I, 1)).to(torch.bfloat16)
    w = torch.from_numpy(v[:, 3].astype(np.float32))
    assert np.array_equal(H1.double().numpy()[:, [0, I]], v[:, :2]) and np.array_equal(G.double().numpy()[:, 0], v[:, 2])
    got = w4.w4_silu_mul_bwd(H1.to(dev()), G.to(dev()), weights=w.to(dev()))
    dh, a, _, _ = train.silu_mul_bwd(H1.double().numpy(), G.double().numpy(), v[:, 3])
    # the sigmoid and each product are good to a few units in the last place of fp32; 1 + g (1 - s)
    # does not cancel at these gates; results below 2^-126 are rounded to steps of 2^-133
    units = 16 * 2.0 ** -24
    for name, y, want in (("dH1", got[0], dh), ("A", got[1], a)):
        y = y.double().cpu().numpy()
        for r, row in enumerate(rows):
            if name == "A":
                parts = [("A", slice(0, I))]
            else:
                parts = [("dg", slice(0, I)), ("du", slice(I, 2 * I))]
            for what, at in parts:
                x, t = y[r, at], want[r, at]
                assert np.isfinite(t).all() and (np.abs(t) < 2.0 ** 127).all()
                tol = (HALF + units) * np.abs(t) + 2.0 ** -126 * (np.abs(t) < 2.0 ** -126) + TINY
                assert (np.abs(x - t) <= tol).all(), f"{what} of {row}: {x[0]} for {t[0]}"


# ------------------------------------------------------------ rows that are not finite --

# the tile kernels (few columns, and sums in parts) and the runs of tiles
@pytest.mark.parametrize("T,k,E,N,K", [(300, 2, 8, 72, 144), (1500, 2, 6, 520, 1040), (96, 2, 32, 1032, 1040),
                                       (4000, 1, 4, 64, 144)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("side", ["gate_up", "down"])
def test_checkpoint_row_that_is_not_finite(T, k, E, N, K, value, side):
    """The first row of X holds a value that is not finite, so that its 128 codes and their scale
    are NaN: only the gradients of the experts that the row goes to may see it."""
    say(f"checkpoint row not finite T={T} k={k} E={E} N={N} K={K} {value} {side}")
    ids = spread(T, k, E)
    dd, dx = (1, k) if side == "gate_up" else (k, 1)
    used = set(ids[0]) if side == "gate_up" else {ids[0, 0]}
    dY, X = normal((T * k // dd, N), 1).to(dev()), normal((T * k // dx, K), 2).to(dev())
    B = w4.w4_bf16_pick_block_size(T, k, E)
    plan = w4.moe_align_block_size(up(ids), E, B)

    def grad():
        X8, SX = w4.w8_quantize_rows(X)
        return w4.w4_bf16_moe_wgrad(dY, X8, *plan, E, T, k, B, dd, dx, SX=SX)
    clean = grad()
    X[0, 5] = value
    got = grad()
    for e in range(E):
        if e in used:
            assert torch.equal(got[e][:, 128:], clean[e][:, 128:]), e
            assert bool(got[e][:, :128].isnan().all()), e
        else:
            assert torch.equal(got[e], clean[e]), e


def test_layer_of_checkpoints_with_a_token_that_is_not_finite():
    """A token that is not finite reaches the gradients of its own experts only."""
    T, k, E, H, I = 70, 2, 8, 128, 64
    ids = spread(T, k, E)
    w = torch.full((T, k), 0.5, device=dev())
    X, gu, dn = normal((T, H), 1).to(dev()), normal((E, 2 * I, H), 2, 0.2).to(dev()), normal((E, H, I), 3, 0.2).to(dev())
    dO = normal((T, H), 4).to(dev())
    dO[0] = 0

    def grads():
        leaves = [t.clone().requires_grad_() for t in (X, gu, dn)]
        out = moe.moe_train(leaves[0], up(ids), w, *leaves[1:], checkpoint=True)
        return torch.autograd.grad(out, leaves, dO)
    clean = grads()
    X[0, 3] = float("nan")
    got = grads()
    others = [e for e in range(E) if e not in ids[0]]
    assert torch.equal(got[0][1:], clean[0][1:])
    for a, b in zip(got[1:], clean[1:]):
        assert torch.equal(a[others], b[others])


# ---------------------------------------------------- how gradients come and go --

def linear_case(kind, shape, N, seed=0):
    X, W = normal((*shape, 64), seed + 1).to(dev()).requires_grad_(), normal((N, 64), seed + 2).to(dev()).requires_grad_()
    call = w8_linear if kind == "w8" else qat_linear
    return X, W, lambda x, w: call(x, w, checkpoint=True)


def moe_case(T=40, k=2, E=4, H=64, I=32, seed=0, **kw):
    ids = up(spread(T, k, E))
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(seed)).to(dev()).requires_grad_()
    X, gu, dn = (normal(s, seed + i, sigma).to(dev()).requires_grad_()
                 for i, (s, sigma) in enumerate((((T, H), 1.0), ((E, 2 * I, H), 0.2), ((E, H, I), 0.2))))
    return (X, w, gu, dn), lambda X, w, gu, dn: moe.moe_train(X, ids, w, gu, dn, checkpoint=True, **kw)


@pytest.mark.parametrize("layer", ["moe", "moe_int4", "w8", "int4"])
def test_gradients_of_every_form(layer):
    """Broadcast, transposed and fp32 gradients are those of the same values laid out plainly; a
    graph can be walked twice."""
    if layer.startswith("moe"):
        leaves, f = moe_case(int4="int4" in layer)
    else:
        *leaves, f = linear_case(layer, (2, 20), 64)
    y = f(*leaves)
    plain = lambda g: torch.autograd.grad(y, leaves, g.contiguous(), retain_graph=True)
    for z, g in ((y.sum(), torch.ones_like(y)), (y.transpose(0, -1).reshape(-1)[::2].sum(), None),
                 (y.float().square().sum(), (2 * y.float()).to(torch.bfloat16))):
        got = torch.autograd.grad(z, leaves, retain_graph=True)
        if g is None:
            g = torch.zeros_like(y.transpose(0, -1)).reshape(-1)
            g[::2] = 1
            g = g.view(y.transpose(0, -1).shape).transpose(0, -1)
        for a, b in zip(got, plain(g)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["w8", "int4"])
def test_linear_checkpoint_graph_replay(kind):
    """Forward and backward from codes in a graph, replayed on new values."""
    X, W, f = linear_case(kind, (300,), 272)
    dY = normal((300, 272), 9).to(dev())

    def step(x, w):
        y = f(x, w)
        return (y, *torch.autograd.grad(y, (x, w), dY))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(X, W)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(X, W)
    for seed in (3, 4, 5):
        with torch.no_grad():
            X.copy_(normal((300, 64), seed))
            W.copy_(normal((272, 64), seed + 10))
            dY.copy_(normal((300, 272), seed + 20))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step(X.detach().clone().requires_grad_(), W.detach().clone().requires_grad_())):
            assert torch.equal(a, b)


def test_linear_checkpoint_of_no_rows_and_of_three_dimensions():
    for kind in ("w8", "int4"):
        X, W, f = linear_case(kind, (0,), 32)
        dX, dW = torch.autograd.grad(f(X, W), (X, W), torch.empty((0, 32), dtype=torch.bfloat16, device=dev()))
        assert dX.shape == X.shape and dW.shape == W.shape and not bool(dW.any())
        X, W, f = linear_case(kind, (3, 7), 32)
        dY = normal((3, 7, 32), 5).to(dev())
        flat = X.detach().reshape(21, 64).requires_grad_()
        for a, b in zip(torch.autograd.grad(f(X, W), (X, W), dY), torch.autograd.grad(f(flat, W), (flat, W), dY.view(21, 32))):
            assert torch.equal(a.reshape(-1), b.reshape(-1))


@pytest.mark.parametrize("R,I", [((1 << 23) + 37, 8), (70000, 16384)])
@pytest.mark.parametrize("codes", [False, True])
def test_silu_mul_bwd_of_many_rows(R, I, codes):
    """More rows than workgroups, and more than 2^31 elements: the last rows are those of a call
    of their own."""
    say(f"silu_mul_bwd of many rows R={R} I={I} codes={codes}")
    g = torch.Generator(device=dev()).manual_seed(1)
    H1 = torch.randn((R, 2 * I), generator=g, device=dev(), dtype=torch.bfloat16)
    G = torch.randn((R, I), generator=g, device=dev(), dtype=torch.bfloat16)
    w, SH = torch.rand(R, generator=g, device=dev()), None
    if codes:
        H1, SH = w4.w8_quantize_rows(H1)
    got = w4.w4_silu_mul_bwd(H1, G, weights=w, SH=SH)
    for rows in (slice(0, 50), slice(R // 2, R // 2 + 50), slice(R - 50, R)):
        few = w4.w4_silu_mul_bwd(H1[rows].clone(), G[rows].clone(), weights=w[rows].clone(), SH=None if SH is None else SH[rows].clone())
        for a, b in zip(got, few):
            assert torch.equal(a[rows], b)
