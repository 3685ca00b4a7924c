"""Training of the routed experts on the GPU: grouped bf16 products in three
directions, the sum over tokens from 8-bit checkpoints, the SwiGLU gradient, and
the layers built of them, against the fp64 oracle.

Tolerances.  An output is rounded once to bf16: half a step, 2^-8 of its value
(bf16 has eight significant bits; below 2^-126 steps are 2^-133).  A sum of n
products carries at most one fp32 rounding a term of the partial sum, which the
terms' magnitudes bound: n 2^-23 of their sum (2^-23, not 2^-24: the matrix unit
need not round to nearest).
"""

import math

import numpy as np
import pytest
import torch

import int4_weight_only_amd as w4
import synth
from gpu_util import canary_bf16, dev, down, down_bits, say, up, CANARY
from int4_weight_only_amd import moe
from int4_weight_only_amd.qat import qat_linear
from int4_weight_only_amd.w8 import w8_linear
from oracle import bf16 as obf
from oracle import train
from oracle import w8 as ow8

pytestmark = pytest.mark.gpu

HALF, TINY = 2.0 ** -8, 2.0 ** -133


def normal(shape, seed, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * sigma).to(torch.bfloat16)


def f64(t):
    return down(t.float()).astype(np.float64)


def codes_f64(x8, sx):
    """fp64 values that a checkpoint stands for."""
    v = ow8.dequant(down(x8.view(torch.uint8)), down(sx.view(torch.uint8)), 1)
    return obf.to_f32(obf.rne(v.astype(np.float32))).astype(np.float64)


def check(got, want, mag, n, what):
    got = f64(got)
    tol = HALF * np.abs(want) + n * 2.0 ** -23 * mag * (1 + HALF) + TINY
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(err / tol):.3g} of the tolerance"


def picks(T, k, E, seed, empty=(), outside=0):
    """ids [T, k] distinct per token, none of the experts in ``empty``; ``outside``
    entries replaced by numbers outside [0, E)."""
    r = np.random.default_rng(seed)
    live = np.array([e for e in range(E) if e not in empty])
    ids = np.stack([r.permutation(live)[:k] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, k), np.int32)
    flat = ids.reshape(-1)
    for i, at in enumerate(r.permutation(flat.size)[:outside]):
        flat[at] = -1 if i % 2 else E + i
    return ids


def plan_of(ids, E, B):
    return w4.moe_align_block_size(up(ids), E, B)


# (T, k, E, N, K, B): one token; sizes below a tile; one past tiles; empty experts; several blocks an
# expert; blocks larger than a tile
PRODUCTS = [(1, 1, 1, 8, 8, 64), (3, 2, 4, 72, 64, 64), (70, 1, 2, 64, 72, 64), (65, 2, 3, 136, 200, 64),
            (200, 2, 3, 264, 136, 128), (300, 3, 5, 520, 328, 256), (257, 1, 1, 256, 512, 256),
            (90, 2, 4, 104, 1000, 192), (600, 1, 2, 320, 192, 1024), (1000, 4, 8, 384, 640, 256),
            (512, 1, 1, 512, 64, 512), (16, 8, 64, 128, 2048, 64)]


@pytest.mark.parametrize("T,k,E,N,K,B", PRODUCTS)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("per_pair", [False, True])
def test_moe_gemm(T, k, E, N, K, B, transposed, per_pair):
    say(f"moe_gemm T={T} k={k} E={E} N={N} K={K} B={B} transposed={transposed} per_pair={per_pair}")
    if not transposed:
        N = N - 3 if N > 8 else 1                     # N need not be a multiple of anything here
    ids = picks(T, k, E, T + N, empty=(1,) if E > k + 1 else (), outside=min(3, T * k // 4))
    div = 1 if per_pair else k
    X = normal((T * k // div, K), 1)
    W = normal((E, K, N) if transposed else (E, N, K), 2, 0.1)
    out = canary_bf16((T * k, N))
    w4.w4_bf16_moe_gemm(X.to(dev()), W.to(dev()), *plan_of(ids, E, B), T, k, B, div, transposed=transposed, out=out)
    want, mag = train.moe_gemm(f64(X), f64(W), ids, div, transposed)
    named = ~np.isnan(want[:, 0])
    assert (down_bits(out)[~named] == CANARY).all()
    check(out[torch.from_numpy(named).to(dev())], want[named], mag[named], K, "Y")


@pytest.mark.parametrize("T,k,E,N,K,B", PRODUCTS)
@pytest.mark.parametrize("side", ["gate_up", "down"])
@pytest.mark.parametrize("codes", [False, True])
def test_moe_wgrad(T, k, E, N, K, B, side, codes):
    say(f"moe_wgrad T={T} k={k} E={E} N={N} K={K} B={B} {side} codes={codes}")
    K = -(-K // 16) * 16
    ids = picks(T, k, E, T + N, empty=(1,) if E > k + 1 else (), outside=min(3, T * k // 4))
    dd, dx = (1, k) if side == "gate_up" else (k, 1)
    dY, X = normal((T * k // dd, N), 1).to(dev()), normal((T * k // dx, K), 2, 3.0).to(dev())
    SX, x = None, f64(X)
    if codes:
        X, SX = w4.w8_quantize_rows(X)
        x = codes_f64(X, SX)
    out = canary_bf16((E, N, K))
    w4.w4_bf16_moe_wgrad(dY, X, *plan_of(ids, E, B), E, T, k, B, dd, dx, SX=SX, out=out)
    want, mag = train.moe_wgrad(f64(dY), x, ids, E, dd, dx)
    check(out, want, mag, T, "dW")


def test_wgrad_without_tokens_is_zero():
    ids = np.zeros((0, 2), np.int32)
    out = canary_bf16((3, 64, 72))
    z = torch.empty((0, 64), dtype=torch.bfloat16, device=dev())
    x = torch.empty((0, 72), dtype=torch.bfloat16, device=dev())
    w4.w4_bf16_moe_wgrad(z, x, *plan_of(ids, 3, 64), 3, 0, 2, 64, 1, 2, out=out)
    assert (down_bits(out) == 0).all()
    out = canary_bf16((64, 72))
    w4.w4_bf16_gemm_tn(z, x, out=out)
    assert (down_bits(out) == 0).all()


@pytest.mark.parametrize("M", [1, 63, 64, 65, 130, 1000, 5000])
@pytest.mark.parametrize("N,K", [(8, 16), (72, 48), (128, 256), (264, 400), (520, 1040)])
@pytest.mark.parametrize("codes", [False, True])
def test_gemm_tn(M, N, K, codes):
    say(f"gemm_tn M={M} N={N} K={K} codes={codes}")
    A, B = normal((M, N), 1).to(dev()), normal((M, K), 2, 2.0).to(dev())
    SB, b = None, f64(B)
    if codes:
        B, SB = w4.w8_quantize_rows(B)
        b = codes_f64(B, SB)
    out = w4.w4_bf16_gemm_tn(A, B, SB=SB)
    want, mag = train.gemm_tn(f64(A), b)
    check(out, want, mag, M, "C")


def test_gemm_tn_of_whole_numbers_is_exact():
    """Sums of small integers are exact in fp32 whatever the order: a wrong index shows."""
    r = np.random.default_rng(3)
    a, b = r.integers(-2, 3, (700, 200)), r.integers(-2, 3, (700, 328))
    t = lambda v: torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16).to(dev())
    got = f64(w4.w4_bf16_gemm_tn(t(a), t(b)))
    np.testing.assert_array_equal(got, f64(torch.from_numpy((a.T @ b).astype(np.float32)).to(torch.bfloat16)))


def test_checkpoint_scales_of_every_exponent():
    """Rows at 2^-130 .. 2^110: the checkpoint's values are taken as they are."""
    M, K = 64, 256
    X = normal((M, K), 5) * torch.exp2(torch.linspace(-126, 110, M)).to(torch.bfloat16)[:, None]
    X[7] = 0
    X8, SX = w4.w8_quantize_rows(X.to(dev()))
    eye = torch.eye(M, dtype=torch.bfloat16, device=dev())
    got = f64(w4.w4_bf16_gemm_tn(eye, X8, SB=SX))
    want = codes_f64(X8, SX)
    normal_ = np.abs(want) >= 2.0 ** -126
    np.testing.assert_array_equal(got[normal_], want[normal_])
    assert (np.abs(got - want)[~normal_] <= 2.0 ** -126).all()


def test_values_of_other_experts_and_skipped_pairs_do_not_reach_a_result():
    """NaN and Inf in rows of one expert, of skipped pairs, and behind a segment."""
    T, k, E, N, K, B = 130, 2, 4, 72, 80, 64
    ids = picks(T, k, E, 9, outside=4)
    flat = ids.reshape(-1)
    X, dY = normal((T * k, K), 1), normal((T * k, N), 2)
    W = normal((E, N, K), 3, 0.1)
    bad = (flat == 2) | (flat < 0) | (flat >= E)
    clean = train.moe_gemm(f64(X), f64(W), ids, 1)
    grad = train.moe_wgrad(f64(dY), f64(X), ids, E, 1, 1)
    X[torch.from_numpy(bad)] = float("nan")
    dY[torch.from_numpy(bad)] = float("inf")
    W[2] = float("nan")
    p = plan_of(ids, E, B)
    Y = w4.w4_bf16_moe_gemm(X.to(dev()), W.to(dev()), *p, T, k, B, 1)
    good = ~bad
    check(Y[torch.from_numpy(good).to(dev())], clean[0][good], clean[1][good], K, "Y")
    dW = w4.w4_bf16_moe_wgrad(dY.to(dev()), X.to(dev()), *p, E, T, k, B, 1, 1)
    for e in (0, 1, 3):
        check(dW[e], grad[0][e], grad[1][e], T, f"dW[{e}]")
    # a NaN of a used row does reach it
    X2 = normal((T, K), 4)
    X2[5, 3] = float("nan")
    e = ids[5][(ids[5] >= 0) & (ids[5] < E)][0]
    dW = w4.w4_bf16_moe_wgrad(normal((T * k, N), 2).to(dev()), X2.to(dev()), *p, E, T, k, B, 1, k)
    assert torch.isnan(dW[int(e), :, 3]).all() and not torch.isnan(dW[:, :, :3]).any()


def test_same_expert_twice_in_a_token():
    T, k, E, N, K, B = 40, 3, 2, 64, 64, 64
    ids = np.random.default_rng(0).integers(0, E, (T, k)).astype(np.int32)
    dY, X = normal((T * k, N), 1), normal((T, K), 2)
    dW = w4.w4_bf16_moe_wgrad(dY.to(dev()), X.to(dev()), *plan_of(ids, E, B), E, T, k, B, 1, k)
    want, mag = train.moe_wgrad(f64(dY), f64(X), ids, E, 1, k)
    check(dW, want, mag, T * k, "dW")


# ------------------------------------------------------------------- SwiGLU --

def check_swiglu(h, G, w, got, I):
    """The sigmoid and its remainder are good to a few units in the last place: 16 2^-24 of each
    result, and of the terms 1 and g (1 - s) where they cancel."""
    dh, a, dw, mag = train.silu_mul_bwd(h, G, w)
    g, u = np.split(h, 2, axis=1)
    ww = np.ones(h.shape[0]) if w is None else w
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-g))
    units = 16 * 2.0 ** -24
    cancel = np.abs(ww[:, None] * G * u * s) * (1 + np.abs(g)) * units
    tol = HALF * np.abs(dh) * (1 + units) + units * np.abs(dh) + TINY
    tol[:, :I] += cancel
    err = np.abs(f64(got[0]) - dh)
    assert (err <= tol).all(), f"dH1: worst {np.max(err / tol):.3g} of the tolerance"
    err = np.abs(f64(got[1]) - a)
    tol = (HALF + 2 * units) * np.abs(a) + TINY
    assert (err <= tol).all(), f"A: worst {np.max(err / tol):.3g} of the tolerance"
    err = np.abs(down(got[2]).astype(np.float64) - dw)
    tol = (I + 32) * 2.0 ** -24 * mag + I * 2.0 ** -149
    assert (err <= tol).all(), f"dw: worst {np.max(err / tol):.3g} of the tolerance"


@pytest.mark.parametrize("R,I", [(1, 8), (3, 16), (64, 136), (257, 2000), (1000, 64), (5, 2048), (7, 4104), (2, 20480)])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_silu_mul_bwd(R, I, codes, weighted):
    say(f"silu_mul_bwd R={R} I={I} codes={codes} weighted={weighted}")
    H1, G = normal((R, 2 * I), 1, 3.0).to(dev()), normal((R, I), 2).to(dev())
    SH, h = None, f64(H1)
    if codes:
        H1, SH = w4.w8_quantize_rows(H1)
        h = codes_f64(H1, SH)
    w = torch.rand(R, generator=torch.Generator().manual_seed(3)).to(dev()) if weighted else None
    got = w4.w4_silu_mul_bwd(H1, G, weights=w, SH=SH)
    check_swiglu(h, f64(G), down(w).astype(np.float64) if weighted else None, got, I)


def test_silu_mul_bwd_far_gates():
    """Gates of -200 .. 200, with factors that bring results back where the sigmoid
    alone is below fp32's range."""
    I = 808
    g = torch.linspace(-200, 200, I).to(torch.bfloat16)
    for su, sg in ((1.0, 1.0), (2.0 ** 100, 1.0), (1.0, 2.0 ** 100), (2.0 ** 60, 2.0 ** 40)):
        H1 = torch.cat([g, normal((I,), 1) * su])[None].to(torch.bfloat16).contiguous()
        G = (normal((1, I), 2) * sg).to(torch.bfloat16)
        got = w4.w4_silu_mul_bwd(H1.to(dev()), G.to(dev()))
        dh, a, _, _ = train.silu_mul_bwd(f64(H1), f64(G))
        for name, y, want in (("dH1", f64(got[0]), dh), ("A", f64(got[1]), a)):
            ok = np.abs(want) < 2.0 ** 127          # larger ones round to infinity
            gg = np.concatenate([f64(H1)[:, :I]] * (want.shape[1] // I), 1)
            # 1 + g (1 - s) cancels near g = -1.28; relative elsewhere
            tol = (HALF + 2.0 ** -18) * np.abs(want) + 2.0 ** -126
            tol = np.where(np.abs(gg + 1.2785) < 0.5, tol + 2.0 ** -18 * np.max(np.abs(want[np.abs(gg) < 3]), initial=0), tol)
            err = np.abs(y - want)
            assert (err[ok] <= tol[ok]).all(), f"{name} su={su} sg={sg}: {np.max(err[ok] / tol[ok])}"


def test_silu_mul_bwd_empty_and_given_outputs():
    G = torch.empty((4, 0), dtype=torch.bfloat16, device=dev())
    H1 = torch.empty((4, 0), dtype=torch.bfloat16, device=dev())
    dw = torch.full((4,), 7.0, device=dev())
    w4.w4_silu_mul_bwd(H1, G, dw=dw)
    assert (down(dw) == 0).all()
    w4.w4_silu_mul_bwd(torch.empty((0, 64), dtype=torch.bfloat16, device=dev()),
                       torch.empty((0, 32), dtype=torch.bfloat16, device=dev()))
    H1, G = normal((5, 64), 1).to(dev()), normal((5, 32), 2).to(dev())
    w = torch.rand((5, 1), device=dev())
    one = w4.w4_silu_mul_bwd(H1, G, weights=w)
    outs = (canary_bf16((5, 64)), canary_bf16((5, 32)), torch.zeros(5, device=dev()))
    two = w4.w4_silu_mul_bwd(H1, G, weights=w, dH1=outs[0], A=outs[1], dw=outs[2])
    assert all(a is b for a, b in zip(two, outs))
    assert all(torch.equal(a, b) for a, b in zip(one, two))


# ------------------------------------------------------------------- layers --

def layer_case(T, k, E, H, I, seed=0, outside=0):
    ids = up(picks(T, k, E, seed, outside=outside))
    w = (torch.rand((T, k), generator=torch.Generator().manual_seed(seed)) + 0.1).to(dev())
    X, gu = normal((T, H), seed + 1).to(dev()), normal((E, 2 * I, H), seed + 2, 0.2).to(dev())
    return ids, w, X, gu, normal((E, H, I), seed + 3, 0.2).to(dev()), normal((T, H), seed + 4).to(dev())


def rounded(x):
    return obf.to_f32(obf.rne(np.nan_to_num(x).astype(np.float32))).astype(np.float64)


def near(got, want, share, what):
    """Chains of rounded stages: a stage's half step turns a few roundings of the next one over, so
    an output is within ``share`` of the tensor's root mean square, beside its own rounding."""
    got = f64(got)
    rms = np.sqrt((want ** 2).mean())
    err = np.abs(got - want)
    tol = HALF * np.abs(want) + share * rms
    assert (err <= tol).all(), f"{what}: worst {np.max(err / tol):.3g} of the tolerance"


@pytest.mark.parametrize("T,k,E,H,I", [(1, 1, 1, 32, 32), (5, 2, 3, 64, 32), (70, 2, 4, 128, 96), (300, 4, 8, 256, 160)])
@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("checkpoint", [False, True])
def test_moe_train(T, k, E, H, I, int4, checkpoint):
    say(f"moe_train T={T} k={k} E={E} H={H} I={I} int4={int4} checkpoint={checkpoint}")
    ids, w, X, gu, dn, dO = layer_case(T, k, E, H, I, T)
    leaves = [t.clone().requires_grad_() for t in (X, w, gu, dn)]
    out = moe.moe_train(leaves[0], ids, *leaves[1:], int4=int4, checkpoint=checkpoint)
    grads = torch.autograd.grad(out, leaves, dO)
    fq = lambda W: w4.w4_fake_quant(W.view(-1, W.shape[2])).view(W.shape) if int4 else W
    Wu, Wd = f64(fq(gu)), f64(fq(dn))
    want, h, _, _ = train.layer(f64(X), down(ids), f64(w), Wu, Wd, rounded)
    # the products' own roundings: two stages of up to eight bits before each output, of which a few
    # in a hundred turn over (fp32 sums of K terms); four half steps of the output's scale cover it
    near(out, want, 4 * HALF, "out")
    x = f64(X)
    if checkpoint:
        x = codes_f64(*w4.w8_quantize_rows(X))
        hb = torch.from_numpy(h.astype(np.float32)).to(torch.bfloat16).to(dev())
        h = codes_f64(*w4.w8_quantize_rows(hb))
    ref = train.layer_bwd(x, h, down(ids), f64(w), Wu, Wd, f64(dO), rounded)
    # with a checkpoint a half step of h that turns over moves a code by a step of its own (2^-3):
    # rare, and one of I terms
    share = 4 * HALF if not checkpoint else 2.0 ** -4
    for name, g, r in zip(("dX", "dw", "dgate_up", "ddown"), grads, ref):
        near(g, r, share, name)


def test_int4_layer_is_the_served_layer():
    """Output of the training forward and of moe_forward on the same codes: equal bits."""
    T, k, E, H, I = 100, 2, 4, 128, 96
    ids, w, X, gu, dn, _ = layer_case(T, k, E, H, I)
    out = moe.moe_train(X, ids, w, gu, dn, int4=True)
    q = lambda W: moe.quantize_experts(E, W.shape[1], W.shape[2], lambda e: W[e], dev())
    B = w4.w4_bf16_pick_block_size(T, k, E)
    assert torch.equal(out, moe.moe_forward(X, ids, w, q(gu), q(dn), B=B)[0])
    assert torch.equal(out, moe.moe_train(X, ids, w, gu, dn, int4=True, checkpoint=True))


@pytest.mark.parametrize("checkpoint", [False, True])
def test_each_gradient_alone_is_the_same(checkpoint):
    ids, w, X, gu, dn, dO = layer_case(40, 2, 4, 64, 32)
    base = (X, w, gu, dn)

    def grads(wanted):
        leaves = [t.clone().requires_grad_(i in wanted) for i, t in enumerate(base)]
        out = moe.moe_train(leaves[0], ids, *leaves[1:], checkpoint=checkpoint)
        return torch.autograd.grad(out, [leaves[i] for i in wanted], dO)
    all_ = grads((0, 1, 2, 3))
    for i in range(4):
        assert torch.equal(grads((i,))[0], all_[i]), i
    for pair in ((0, 3), (1, 2)):
        for i, g in zip(pair, grads(pair)):
            assert torch.equal(g, all_[i])


def test_moe_train_follows_differences():
    """<gradient, direction> against the change of the fp64 layer along it."""
    T, k, E, H, I = 30, 2, 3, 64, 64
    ids, w, X, gu, dn, dO = layer_case(T, k, E, H, I, 11)
    leaves = [t.clone().requires_grad_() for t in (X, w, gu, dn)]
    grads = torch.autograd.grad(moe.moe_train(leaves[0], ids, *leaves[1:]), leaves, dO)
    args = [f64(t) for t in (X, w, gu, dn)]
    f = lambda a: (train.layer(a[0], down(ids), *a[1:])[0] * f64(dO)).sum()
    for i, g in enumerate(grads):
        # along the gradient itself: a wrong scale or a missing term shows whole
        d = f64(g)
        eps = 1e-5 / np.sqrt((d ** 2).mean())
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + eps * d, args[i] - eps * d
        slope = (f(hi) - f(lo)) / (2 * eps)
        # every stage rounds to bf16: half steps at random in thousands of terms, and one eighth of a
        # per cent of systematic room
        assert abs(slope - (d * d).sum()) <= 2.0 ** -7 * (d * d).sum(), i


def test_moe_train_of_no_tokens():
    ids, w, X, gu, dn, dO = layer_case(0, 2, 4, 64, 32)
    leaves = [t.clone().requires_grad_() for t in (X, w, gu, dn)]
    for kw in (dict(), dict(int4=True, checkpoint=True)):
        out = moe.moe_train(leaves[0], ids, *leaves[1:], **kw)
        assert out.shape == (0, 64)
        for g, t in zip(torch.autograd.grad(out, leaves, dO), leaves):
            assert g.shape == t.shape and (down(g.float()) == 0).all()


def test_router_and_experts_together():
    """The scored router's gradient through the layer, as a training step uses them."""
    T, k, E, H, I = 60, 2, 8, 64, 32
    _, _, X, gu, dn, dO = layer_case(T, k, E, H, I, 5)
    logits = normal((T, E), 9).float().to(dev()).requires_grad_()
    gu.requires_grad_()
    ids, w = moe.route_scored(logits, k, sigmoid=True)
    out = moe.moe_train(X, ids, w, gu, dn, checkpoint=True)
    dl, dgu = torch.autograd.grad(out, (logits, gu), dO)
    w2 = w.detach().clone().requires_grad_()
    dw, dgu2 = torch.autograd.grad(moe.moe_train(X, ids, w2, gu, dn, checkpoint=True), (w2, gu), dO)
    assert torch.equal(dgu, dgu2)
    assert torch.equal(dl, w4.w4_moe_route_scored_bwd(logits.detach(), ids, w.detach(), dw, sigmoid=True))


def test_moe_train_refusals():
    ids, w, X, gu, dn, dO = layer_case(8, 2, 4, 64, 32)
    with pytest.raises(ValueError):
        moe.moe_train(X, ids, w, gu[:, :-1], dn)
    with pytest.raises(ValueError):
        moe.moe_train(X, ids[:4], w, gu, dn)
    with pytest.raises(ValueError):
        moe.moe_train(X, ids, w[:, :1], gu, dn)
    with pytest.raises(TypeError):
        moe.moe_train(X, ids, w.bfloat16(), gu, dn)
    with pytest.raises(ValueError):
        moe.moe_train(X, ids, w, gu[:, :48].contiguous(), dn[:, :, :24].contiguous(), int4=True)
    with pytest.raises(ValueError):
        moe.moe_train(X[:, ::2], ids, w, gu, dn)
    Xg = X.clone().requires_grad_()
    out = moe.moe_train(Xg, ids, w, gu, dn)
    g = torch.autograd.grad(out, Xg, dO, create_graph=True)[0]
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.sum(), Xg)


def test_no_grad_keeps_nothing():
    ids, w, X, gu, dn, _ = layer_case(8, 2, 4, 64, 32)
    gu.requires_grad_()
    with torch.no_grad():
        assert not moe.moe_train(X, ids, w, gu, dn, checkpoint=True).requires_grad


@pytest.mark.parametrize("M,N,K", [(1, 16, 32), (70, 64, 96), (333, 264, 160)])
@pytest.mark.parametrize("kind", ["w8", "int4"])
def test_linear_checkpoint(M, N, K, kind):
    say(f"linear checkpoint M={M} N={N} K={K} {kind}")
    N = -(-N // 16) * 16
    layer = w8_linear if kind == "w8" else qat_linear
    X, W, dY = normal((M, K), 1).to(dev()), normal((N, K), 2, 0.1).to(dev()), normal((M, N), 3).to(dev())
    X.requires_grad_(), W.requires_grad_()
    plain = layer(X, W)
    kept = layer(X, W, checkpoint=True)
    assert torch.equal(plain, kept)
    dX, _ = torch.autograd.grad(plain, (X, W), dY)
    dXc, dWc = torch.autograd.grad(kept, (X, W), dY)
    assert torch.equal(dX, dXc)
    want, mag = train.gemm_tn(f64(dY), codes_f64(*w4.w8_quantize_rows(X.detach())))
    check(dWc, want, mag, M, "dW")


def test_checkpoint_halves_what_a_layer_keeps():
    X, W = normal((2048, 1024), 1).to(dev()), normal((64, 1024), 2).to(dev()).requires_grad_()
    for layer in (w8_linear, qat_linear):
        saved = []
        for c in (False, True):
            Y = layer(X, W, checkpoint=c)
            saved.append(sum(t.numel() * t.element_size() for t in Y.grad_fn.saved_tensors if t is not None
                             and t.shape[0] == X.shape[0]))
            del Y
        assert saved[1] <= saved[0] * 0.51


# ---------------------------------------------------- streams, graphs, order --

def step(leaves, ids, dO, **kw):
    out = moe.moe_train(leaves[0], ids, *leaves[1:], **kw)
    return (out, *torch.autograd.grad(out, leaves, dO))


@pytest.mark.parametrize("int4", [False, True])
def test_graph_replays(int4):
    ids, w, X, gu, dn, dO = layer_case(90, 2, 4, 128, 64)
    leaves = [t.clone().requires_grad_() for t in (X, w, gu, dn)]
    kw = dict(int4=int4, checkpoint=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step(leaves, ids, dO, **kw)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(leaves, ids, dO, **kw)
    for seed in (1, 2, 3):
        new = layer_case(90, 2, 4, 128, 64, seed)
        with torch.no_grad():
            for t, v in zip((ids, leaves[1], leaves[0], leaves[2], leaves[3], dO), new):
                t.copy_(v)
        g.replay()
        torch.cuda.synchronize()
        fresh = [t.detach().clone().requires_grad_() for t in leaves]
        for a, b in zip(got, step(fresh, ids, dO, **kw)):
            assert torch.equal(a, b)


def test_another_stream_and_twice_the_same_bits():
    ids, w, X, gu, dn, dO = layer_case(500, 2, 4, 256, 128)
    leaves = [t.clone().requires_grad_() for t in (X, w, gu, dn)]
    one = step(leaves, ids, dO)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    results = []
    for s in streams:
        with torch.cuda.stream(s):
            results.append(step([t.detach().clone().requires_grad_() for t in leaves], ids, dO))
    torch.cuda.synchronize()
    for r in results:
        for a, b in zip(one, r):
            assert torch.equal(a, b)


# ---------------------------------------------------------- larger sizes --
# Sizes at which each shape of tile is chosen, against fp64 sums on the GPU (the
# oracle's loops in another place).

def check_large(got, want, mag, n, what):
    tol = HALF * want.abs() + n * 2.0 ** -23 * mag * (1 + HALF) + TINY
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), f"{what}: worst {float((err / tol).max()):.3g} of the tolerance"


def stored(x, s):
    if s is None:
        return x.double()
    v = torch.exp2(s.view(torch.uint8).double() - 127).repeat_interleave(128, 1)[:, : x.shape[1]]
    return x.float().double() * v


@pytest.mark.parametrize("M,N,K", [(700, 4096, 4096), (2050, 2304, 4112), (1500, 1024, 2064), (900, 1096, 1040),
                                   (2048, 512, 768), (4100, 264, 272), (20000, 64, 80)])
@pytest.mark.parametrize("codes", [False, True])
def test_large_gemm_tn(M, N, K, codes):
    say(f"large gemm_tn M={M} N={N} K={K} codes={codes}")
    A, B, SB = normal((M, N), 1).to(dev()), normal((M, K), 2).to(dev()), None
    if codes:
        B, SB = w4.w8_quantize_rows(B)
    b = stored(B, SB)
    check_large(w4.w4_bf16_gemm_tn(A, B, SB=SB), A.double().t() @ b, A.double().abs().t() @ b.abs(), M, "C")


@pytest.mark.parametrize("T,k,E,N,K", [(2000, 2, 4, 4096, 2048), (1500, 4, 16, 1040, 2064), (3000, 2, 8, 520, 784),
                                       (700, 4, 8, 256, 512), (900, 8, 32, 136, 272), (4000, 1, 2, 64, 64),
                                       (300, 2, 64, 1408, 1024)])
@pytest.mark.parametrize("codes", [False, True])
def test_large_grouped(T, k, E, N, K, codes):
    """The three directions on skewed experts."""
    say(f"large grouped T={T} k={k} E={E} N={N} K={K} codes={codes}")
    g = torch.Generator().manual_seed(4)
    lg = torch.randn((T, E), generator=g)
    lg[:, : max(1, E // 8)] += 1.5
    ids = torch.topk(lg, k, 1).indices.to(torch.int32).to(dev())
    B = w4.w4_bf16_pick_block_size(T, k, E)
    p = w4.moe_align_block_size(ids, E, B)
    X, dY, SX = normal((T, K), 1).to(dev()), normal((T * k, N), 2).to(dev()), None
    W = normal((E, N, K), 3, 0.05).to(dev())
    flat = ids.reshape(-1)
    if not codes:
        Y = w4.w4_bf16_moe_gemm(X, W, *p, T, k, B, k)
        dX = w4.w4_bf16_moe_gemm(dY, W, *p, T, k, B, 1, transposed=True)
        few = w4.w4_bf16_moe_gemm(X, W, *w4.moe_align_block_size(ids, E, 64), T, k, 64, k)
    else:
        X, SX = w4.w8_quantize_rows(X)
    dW = w4.w4_bf16_moe_wgrad(dY, X, *p, E, T, k, B, 1, k, SX=SX)
    x = stored(X, SX)
    for e in range(E):
        f = torch.nonzero(flat == e)[:, 0]
        xe, ye, we = x[f // k], dY[f].double(), W[e].double()
        check_large(dW[e], ye.t() @ xe, ye.abs().t() @ xe.abs(), T, f"dW[{e}]")
        if not codes:
            check_large(Y[f], xe @ we.t(), xe.abs() @ we.abs().t(), K, f"Y of {e}")
            check_large(few[f], xe @ we.t(), xe.abs() @ we.abs().t(), K, f"Y of {e}, small blocks")
            check_large(dX[f], ye @ we, ye.abs() @ we.abs(), N, f"dX of {e}")


# -------------------------------------------------- sums in parts, workspaces --

@pytest.mark.parametrize("M,N,K", [(8192, 64, 64), (1024, 8, 16), (3000, 200, 136), (513, 64, 1040)])
@pytest.mark.parametrize("codes", [False, True])
def test_gemm_tn_in_parts(M, N, K, codes, monkeypatch):
    K = -(-K // 16) * 16 if codes else K              # rows of codes are whole 16-byte pieces
    say(f"gemm_tn in parts M={M} N={N} K={K} codes={codes}")
    size = w4.w4_bf16_gemm_tn_workspace(M, N, K)
    assert size % (N * K) == 0                        # 0: the rule takes these whole either way
    A, B, SB = normal((M, N), 1).to(dev()), normal((M, K), 2).to(dev()), None
    if codes:
        B, SB = w4.w8_quantize_rows(B)
    b = stored(B, SB)
    want, mag = A.double().t() @ b, A.double().abs().t() @ b.abs()
    ws = torch.full((size,), float("nan"), device=dev())
    parts = w4.w4_bf16_gemm_tn(A, B, SB=SB, workspace=ws)
    check_large(parts, want, mag, M, "parts")
    assert torch.equal(parts, w4.w4_bf16_gemm_tn(A, B, SB=SB))
    monkeypatch.setattr(w4, "w4_bf16_gemm_tn_workspace", lambda *a: 0)        # a caller without one
    check_large(w4.w4_bf16_gemm_tn(A, B, SB=SB), want, mag, M, "whole")
    monkeypatch.undo()
    if size:
        with pytest.raises(ValueError):
            w4.w4_bf16_gemm_tn(A, B, SB=SB, workspace=ws[:-1])
        with pytest.raises(TypeError):
            w4.w4_bf16_gemm_tn(A, B, SB=SB, workspace=ws.bfloat16())


@pytest.mark.parametrize("T,k,E,N,K", [(1, 1, 1, 4096, 4096), (3, 2, 4, 264, 2048), (5, 1, 2, 8, 8192)])
@pytest.mark.parametrize("transposed", [False, True])
def test_moe_gemm_in_parts(T, k, E, N, K, transposed, monkeypatch):
    say(f"moe_gemm in parts T={T} k={k} E={E} N={N} K={K} transposed={transposed}")
    N = N if transposed else N - 3
    B = 64
    size = w4.w4_bf16_moe_gemm_workspace(T, k, E, N, K, B)
    assert size or K < 4096
    ids = picks(T, k, E, 3, outside=1 if T > 2 else 0)
    X, W = normal((T, K), 1), normal((E, K, N) if transposed else (E, N, K), 2, 0.1)
    want, mag = train.moe_gemm(f64(X), f64(W), ids, k, transposed)
    named = ~np.isnan(want[:, 0])
    args = (X.to(dev()), W.to(dev()), *plan_of(ids, E, B), T, k, B, k)
    for parts in (True, False):
        out = canary_bf16((T * k, N))
        if parts:
            ws = torch.full((size,), float("nan"), device=dev())
            w4.w4_bf16_moe_gemm(*args, transposed=transposed, out=out, workspace=ws)
        else:
            monkeypatch.setattr(w4, "w4_bf16_moe_gemm_workspace", lambda *a: 0)
            w4.w4_bf16_moe_gemm(*args, transposed=transposed, out=out)
        assert (down_bits(out)[~named] == CANARY).all()
        check(out[torch.from_numpy(named).to(dev())], want[named], mag[named], K, f"parts={parts}")


def test_moe_wgrad_in_parts():
    """Parts of experts with many, few and no pairs."""
    T, k, E, N, K, B = 4000, 1, 3, 72, 80, 256
    size = w4.w4_bf16_moe_wgrad_workspace(T, k, E, N, K)
    assert size > 0
    ids = np.zeros((T, k), np.int32)
    ids[:70] = 2
    dY, X = normal((T, N), 1), normal((T, K), 2)
    out = canary_bf16((E, N, K))
    ws = torch.full((size,), float("nan"), device=dev())
    w4.w4_bf16_moe_wgrad(dY.to(dev()), X.to(dev()), *plan_of(ids, E, B), E, T, k, B, 1, 1, out=out, workspace=ws)
    want, mag = train.moe_wgrad(f64(dY), f64(X), ids, E, 1, 1)
    check(out, want, mag, T, "dW")
    assert (down_bits(out)[1] == 0).all()


def test_graph_replays_of_products_in_parts():
    A, B = normal((4096, 64), 1).to(dev()), normal((4096, 72), 2).to(dev())
    X, W = normal((2, 4096), 3).to(dev()), normal((1, 512, 4096), 4).to(dev())
    ids = torch.zeros((2, 1), dtype=torch.int32, device=dev())
    assert w4.w4_bf16_gemm_tn_workspace(4096, 64, 72) and w4.w4_bf16_moe_gemm_workspace(2, 1, 1, 512, 4096, 64)

    def run():
        return (w4.w4_bf16_gemm_tn(A, B),
                w4.w4_bf16_moe_gemm(X, W, *w4.moe_align_block_size(ids, 1, 64), 2, 1, 64, 1))
    run()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):                                # two graphs, each with workspaces of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, run()))
    for seed in (5, 6, 7):
        A.copy_(normal((4096, 64), seed))
        X.copy_(normal((2, 4096), seed))
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, got in graphs:
            for a, b in zip(got, run()):
                assert torch.equal(a, b)


# ------------------------------------------------------------- wide operands --

def test_operands_of_two_gib_and_more():
    """Rows past 2^31 bytes: the last rows' values are where they belong."""
    T, K, N, E, B = (1 << 17) + 70, 8192, 64, 2, 256
    g = torch.Generator(device=dev()).manual_seed(1)
    X = torch.randn((T, K), generator=g, device=dev(), dtype=torch.bfloat16)
    W, dY = normal((E, N, K), 2, 0.05).to(dev()), normal((T, N), 3).to(dev())
    ids = torch.randint(0, E, (T, 1), generator=g, device=dev(), dtype=torch.int32)
    p = w4.moe_align_block_size(ids, E, B)
    Y = w4.w4_bf16_moe_gemm(X, W, *p, T, 1, B, 1)
    rows = torch.cat([torch.arange(0, 40), torch.arange(T - 200, T)]).to(dev())
    e = ids[rows, 0].long()
    x = X[rows].double()
    want = torch.einsum("rk,rnk->rn", x, W.double()[e])
    mag = torch.einsum("rk,rnk->rn", x.abs(), W.double().abs()[e])
    check_large(Y[rows], want, mag, K, "Y")
    cols = slice(0, 64)
    dW = w4.w4_bf16_moe_wgrad(dY, X, *p, E, T, 1, B, 1, 1)
    C = w4.w4_bf16_gemm_tn(dY, X)
    X8, SX = w4.w8_quantize_rows(X)
    C8 = w4.w4_bf16_gemm_tn(dY, X8, SB=SX)
    xc, d = X[:, cols].double(), dY.double()
    for i in range(E):
        f = (ids[:, 0] == i)[:, None]
        check_large(dW[i][:, cols], (d * f).t() @ xc, (d * f).abs().t() @ xc.abs(), T, f"dW[{i}]")
    check_large(C[:, cols], d.t() @ xc, d.abs().t() @ xc.abs(), T, "C")
    x8 = stored(X8[:, :128].contiguous(), SX[:, :1].contiguous())[:, cols]
    check_large(C8[:, cols], d.t() @ x8, d.abs().t() @ x8.abs(), T, "C from codes")


# ---------------------------------------------------------------- short sums --
# Results that are large next to their sums, which a workgroup computes as a run of
# tiles: one stage and several, last tiles of a run and of a row, an expert with most
# of the pairs.

def guarded(shape):
    """bf16 tensor of ``shape`` between canaries, and a check of them."""
    n = math.prod(shape)
    base = canary_bf16((n + 8192,))

    def check_ends():
        bits = down_bits(base)
        assert (bits[:4096] == CANARY).all() and (bits[n + 4096:] == CANARY).all()
    return base[4096:4096 + n].view(shape), check_ends


@pytest.mark.parametrize("T,k,E,N,K,hot", [(1, 1, 1, 2048, 2064, 0), (40, 2, 16, 1408, 1040, 0),
                                           (300, 2, 32, 1032, 784, 0), (200, 4, 32, 648, 2320, 180),
                                           (700, 1, 8, 1536, 1168, 500), (64, 1, 64, 776, 656, 64)])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("side", ["gate_up", "down"])
def test_short_grouped_sums(T, k, E, N, K, hot, codes, side):
    say(f"short grouped sums T={T} k={k} E={E} N={N} K={K} hot={hot} codes={codes} {side}")
    ids = picks(T, k, E, T, empty=(1,) if E > k + 1 else (), outside=min(2, T * k // 8))
    ids[:hot, 0] = 0
    dd, dx = (1, k) if side == "gate_up" else (k, 1)
    dY, X, SX = normal((T * k // dd, N), 1).to(dev()), normal((T * k // dx, K), 2, 3.0).to(dev()), None
    if codes:
        X, SX = w4.w8_quantize_rows(X)
    B = w4.w4_bf16_pick_block_size(T, k, E)
    out, check_ends = guarded((E, N, K))
    w4.w4_bf16_moe_wgrad(dY, X, *plan_of(ids, E, B), E, T, k, B, dd, dx, SX=SX, out=out)
    check_ends()
    x, flat = stored(X, SX), up(ids).reshape(-1)
    for e in range(E):
        f = torch.nonzero(flat == e)[:, 0]
        xe, ye = x[f // dx], dY[f // dd].double()
        check_large(out[e], ye.t() @ xe, ye.abs().t() @ xe.abs(), T, f"dW[{e}]")


@pytest.mark.parametrize("M", [1, 40, 64, 65, 129])
@pytest.mark.parametrize("N,K", [(4096, 4112), (2056, 6160)])
@pytest.mark.parametrize("codes", [False, True])
def test_short_dense_sums(M, N, K, codes):
    say(f"short dense sums M={M} N={N} K={K} codes={codes}")
    A, B, SB = normal((M, N), 1).to(dev()), normal((M, K), 2).to(dev()), None
    if codes:
        B, SB = w4.w8_quantize_rows(B)
    out, check_ends = guarded((N, K))
    w4.w4_bf16_gemm_tn(A, B, SB=SB, out=out)
    check_ends()
    b = stored(B, SB)
    check_large(out, A.double().t() @ b, A.double().abs().t() @ b.abs(), M, "C")


def test_short_sums_of_rows_that_hold_nan():
    """NaN and infinity in rows of other experts and of skipped pairs stay there."""
    T, k, E, N, K = 96, 2, 32, 1032, 1040
    ids = picks(T, k, E, 5, empty=(3,), outside=6)
    dY, X = normal((T * k, N), 1), normal((T * k, K), 2)
    flat = torch.from_numpy(ids.reshape(-1).copy())
    bad = (flat == 7) | (flat < 0) | (flat >= E)
    dY[bad] = float("nan")
    X[bad] = float("inf")
    got = w4.w4_bf16_moe_wgrad(dY.to(dev()), X.to(dev()), *plan_of(ids, E, 64), E, T, k, 64, 1, 1)
    for e in range(E):
        f = torch.nonzero(flat == e)[:, 0]
        if e == 7:
            assert f.numel() and bool(got[e].isnan().all())
            continue
        ye, xe = dY[f].double().to(dev()), X[f].double().to(dev())
        check_large(got[e], ye.t() @ xe, ye.abs().t() @ xe.abs(), T, f"dW[{e}]")


@pytest.mark.parametrize("N,B", [(64, 64), (64, 128), (520, 256)])
@pytest.mark.parametrize("transposed", [False, True])
def test_tiles_with_wide_addresses(N, B, transposed):
    """The last rows of X, past 2^31 bytes, in each tile of the products by rows, and the
    weight gradients of few and of many columns."""
    T, K, E = (1 << 17) + 40, 8208, 2
    say(f"wide addresses N={N} B={B} transposed={transposed}")
    g = torch.Generator(device=dev()).manual_seed(7)
    X = torch.randn((T, K), generator=g, device=dev(), dtype=torch.bfloat16)
    W = normal((E, K, N) if transposed else (E, N, K), 2, 0.05).to(dev())
    ids = torch.randint(0, E, (T, 1), generator=g, device=dev(), dtype=torch.int32)
    p = w4.moe_align_block_size(ids, E, B)
    Y = w4.w4_bf16_moe_gemm(X, W, *p, T, 1, B, 1, transposed=transposed)
    rows = torch.cat([torch.arange(0, 30), torch.arange(T - 150, T)]).to(dev())
    x, w, one = X[rows].double(), W.double(), ids[rows, 0] == 1
    for e in range(E):
        at = one if e else ~one
        we = w[e] if transposed else w[e].t().contiguous()
        check_large(Y[rows[at]], x[at] @ we, x[at].abs() @ we.abs(), K, f"Y of {e}")
    del Y
    dY = normal((T, N), 3).to(dev())
    dW = w4.w4_bf16_moe_wgrad(dY, X, *p, E, T, 1, B, 1, 1)
    cols = slice(K - 24, K)
    xc, d = X[:, cols].double(), dY.double()
    for e in range(E):
        f = (ids[:, 0] == e)[:, None]
        check_large(dW[e][:, cols], (d * f).t() @ xc, (d * f).abs().t() @ xc.abs(), T, f"dW[{e}]")
    X8, SX = w4.w8_quantize_rows(X)
    dW = w4.w4_bf16_moe_wgrad(dY, X8, *p, E, T, 1, B, 1, 1, SX=SX)
    last = K // 128 * 128                             # the last scale's columns
    xc = stored(X8[:, last:].contiguous(), SX[:, K // 128: K // 128 + 1].contiguous())
    for e in range(E):
        f = (ids[:, 0] == e)[:, None]
        check_large(dW[e][:, last:], (d * f).t() @ xc, (d * f).abs().t() @ xc.abs(), T, f"dW[{e}] from codes")
