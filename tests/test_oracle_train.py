"""Pins of the training oracle: textbook loops, and derivatives by differences."""

import numpy as np
import pytest

from oracle import train


def case(T, k, E, H, I, seed=0):
    r = np.random.default_rng(seed)
    ids = np.stack([r.permutation(E)[:k] for _ in range(T)])
    w = r.random((T, k)) + 0.1
    return (r, ids, w, r.standard_normal((T, H)), r.standard_normal((E, 2 * I, H)) * 0.3,
            r.standard_normal((E, H, I)) * 0.3)


def test_products_are_the_loops():
    r, ids, _, X, W, _ = case(5, 2, 4, 3, 2)
    ids[1, 1], ids[4, 0] = -1, 9                          # outside [0, E)
    Y, mag = train.moe_gemm(X, W, ids, 2)
    dY = r.standard_normal((10, 4))
    Yt, _ = train.moe_gemm(dY, W, ids, 1, transposed=True)
    dW, _ = train.moe_wgrad(dY, X, ids, 4, 1, 2)
    want = np.zeros_like(W)
    for t in range(5):
        for j in range(2):
            e, f = ids[t, j], 2 * t + j
            if not 0 <= e < 4:
                assert np.isnan(Y[f]).all() and np.isnan(Yt[f]).all()
                continue
            for n in range(4):
                assert Y[f, n] == pytest.approx(sum(X[t, i] * W[e, n, i] for i in range(3)))
                assert mag[f, n] == pytest.approx(sum(abs(X[t, i] * W[e, n, i]) for i in range(3)))
                for i in range(3):
                    want[e, n, i] += dY[f, n] * X[t, i]
            for i in range(3):
                assert Yt[f, i] == pytest.approx(sum(dY[f, n] * W[e, n, i] for n in range(4)))
    np.testing.assert_allclose(dW, want, rtol=1e-12)
    A, B = r.standard_normal((7, 3)), r.standard_normal((7, 2))
    np.testing.assert_allclose(train.gemm_tn(A, B)[0], np.einsum("mn,mk->nk", A, B), rtol=1e-12)


def test_swiglu_gradient_by_differences():
    r = np.random.default_rng(1)
    h, G, w = r.standard_normal((4, 6)) * 3, r.standard_normal((4, 3)), r.random(4)
    dh, a, dw, _ = train.silu_mul_bwd(h, G, w)
    np.testing.assert_allclose(a, w[:, None] * train.silu_mul(h), rtol=1e-12)
    f = lambda h, w: (w[:, None] * G * train.silu_mul(h)).sum()
    eps = 1e-6
    for i in np.ndindex(h.shape):
        d = np.zeros_like(h)
        d[i] = eps
        assert dh[i] == pytest.approx((f(h + d, w) - f(h - d, w)) / (2 * eps), rel=1e-7, abs=1e-9)
    for i in range(4):
        d = np.zeros_like(w)
        d[i] = eps
        assert dw[i] == pytest.approx((f(h, w + d) - f(h, w - d)) / (2 * eps), rel=1e-7, abs=1e-9)


def test_layer_gradients_by_differences():
    r, ids, w, X, gu, dn = case(4, 2, 3, 3, 2, 2)
    dO = r.standard_normal((4, 3))
    f = lambda X, w, gu, dn: (train.layer(X, ids, w, gu, dn)[0] * dO).sum()
    args = [X, w, gu, dn]
    grads = train.layer_bwd(X, train.layer(X, ids, w, gu, dn)[1], ids, w, gu, dn, dO)
    eps = 1e-6
    for n, g in enumerate(grads):
        assert g.shape == args[n].shape
        for i in np.ndindex(g.shape):
            lo, hi = [a.copy() for a in args], [a.copy() for a in args]
            lo[n][i] -= eps
            hi[n][i] += eps
            assert g[i] == pytest.approx((f(*hi) - f(*lo)) / (2 * eps), rel=1e-6, abs=1e-8)


def test_one_expert_is_the_dense_layer():
    r, ids, _, X, gu, dn = case(6, 1, 1, 4, 3, 3)
    out, h, a, _ = train.layer(X, ids, np.ones((6, 1)), gu, dn)
    g, u = np.split(X @ gu[0].T, 2, axis=1)
    np.testing.assert_allclose(out, (g / (1 + np.exp(-g)) * u) @ dn[0].T, rtol=1e-12)
