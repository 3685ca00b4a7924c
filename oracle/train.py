"""Reference for training the routed experts -- TEST INFRASTRUCTURE ONLY.

Pairs f = t * k + j go to expert ids[t, j]; ids outside [0, E) take no part.
All sums are fp64.  ``*_magnitude`` results are the same sums of absolute
values, which bound what rounding in a sum may cost.
"""

import numpy as np


def _pairs(ids, E):
    flat = np.asarray(ids).reshape(-1)
    return [np.nonzero(flat == e)[0] for e in range(E)]


def moe_gemm(X, W, ids, div, transposed=False):
    """X [T k / div, K], W [E, N, K] (transposed: [E, K, N]) -> (Y [T k, N] with
    NaN in rows of pairs without an expert, magnitude)."""
    E = W.shape[0]
    N = W.shape[2] if transposed else W.shape[1]
    Y = np.full((np.asarray(ids).size, N), np.nan)
    mag = np.full_like(Y, np.nan)
    for e, f in enumerate(_pairs(ids, E)):
        w = W[e] if transposed else W[e].T
        Y[f] = X[f // div] @ w
        mag[f] = np.abs(X[f // div]) @ np.abs(w)
    return Y, mag


def moe_wgrad(dY, X, ids, E, dy_div, x_div):
    """(dW [E, N, K], magnitude)."""
    dW = np.zeros((E, dY.shape[1], X.shape[1]))
    mag = np.zeros_like(dW)
    for e, f in enumerate(_pairs(ids, E)):
        a, b = dY[f // dy_div], X[f // x_div]
        dW[e] = a.T @ b
        mag[e] = np.abs(a).T @ np.abs(b)
    return dW, mag


def gemm_tn(A, B):
    return A.T @ B, np.abs(A).T @ np.abs(B)


def _sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def silu_mul(h):
    g, u = np.split(h, 2, axis=1)
    return g * _sigmoid(g) * u


def silu_mul_bwd(h, dA, w=None):
    """h [R, 2I], dA [R, I], w [R] -> (dH1, A, dw, sum of |dA a|)."""
    g, u = np.split(h, 2, axis=1)
    s = _sigmoid(g)
    w = np.ones(h.shape[0]) if w is None else w
    a = g * s * u
    d = w[:, None] * dA
    return (np.concatenate([d * u * s * (1 + g * (1 - s)), d * g * s], 1), w[:, None] * a,
            (dA * a).sum(1), np.abs(dA * a).sum(1))


def layer(X, ids, w, gate_up, down, bf16=lambda x: x):
    """(out, h, a, h2) of the routed layer; ``bf16`` rounds what the layer stores."""
    T, k = ids.shape
    h = bf16(moe_gemm(X, gate_up, ids, k)[0])
    a = bf16(silu_mul(h))
    h2 = bf16(moe_gemm(a, down, ids, 1)[0])
    return (h2.reshape(T, k, -1) * w[:, :, None]).sum(1), h, a, h2


def layer_bwd(X, h, ids, w, gate_up, down, dO, bf16=lambda x: x):
    """Gradients (X, w, gate_up, down) of ``layer``'s out times dO, from the kept
    X and h."""
    T, k = ids.shape
    E = gate_up.shape[0]
    G = bf16(moe_gemm(dO, down, ids, k, transposed=True)[0])
    dh, a, dw, _ = silu_mul_bwd(h, G, w.reshape(-1))
    dh, a = bf16(dh), bf16(a)
    dX = bf16(moe_gemm(dh, gate_up, ids, 1, transposed=True)[0]).reshape(T, k, -1).sum(1)
    return dX, dw.reshape(T, k), moe_wgrad(dh, X, ids, E, 1, k)[0], moe_wgrad(dO, a, ids, E, k, 1)[0]
