"""The training entry points without a GPU: sizes, refusals of the C ABI
(nothing here reaches the HIP runtime) and of the binding."""

import ctypes

import pytest
import torch

import int4_weight_only_amd as w4
from int4_weight_only_amd import _lib, moe

A16, A4, A2 = (ctypes.c_void_p(0x10000 + o) for o in (0, 4, 2))
OK, NULL, SHAPE, MISALIGNED, UNSUPPORTED = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_pick_block_size(lib):
    for T, k, E, B in ((0, 1, 1, 64), (1, 1, 1, 64), (42, 1, 1, 64), (43, 1, 1, 128), (85, 1, 1, 128),
                       (86, 1, 1, 256), (4096, 8, 384, 128), (1 << 60, 8, 64, 256), (1 << 40, 1 << 30, 1, 256)):
        assert lib.w4_bf16_pick_block_size(T, k, E) == w4.w4_bf16_pick_block_size(T, k, E) == B
    f = lib.w4_bf16_pick_block_size
    assert f(-1, 1, 1) == f(1, 0, 1) == f(1, 1, 0) == 0


def moe_gemm(lib, X=A16, W=A16, s=A4, e=A4, n=A4, Y=A2, T=4, k=2, E=8, N=64, K=64, B=64, div=2, tr=0, ws=None):
    return lib.w4_bf16_moe_gemm(X, W, s, e, n, Y, T, k, E, N, K, B, div, tr, ws, None)


def wgrad(lib, dY=A16, X=A16, SX=None, s=A4, e=A4, n=A4, dW=A16, T=4, k=2, E=8, N=64, K=64, B=64, dd=1, dx=2, ws=None):
    return lib.w4_bf16_moe_wgrad(dY, X, SX, s, e, n, dW, T, k, E, N, K, B, dd, dx, ws, None)


@pytest.mark.parametrize("f", [moe_gemm, wgrad])
def test_grouped_refusals(lib, f):
    for bad in (dict(T=-1), dict(k=0), dict(E=0), dict(N=0), dict(K=0), dict(K=4), dict(B=0), dict(B=16),
                dict(B=96)):
        assert f(lib, **bad) == SHAPE
    for bad in (dict(B=1088), dict(E=1025), dict(N=(1 << 22) + 8), dict(K=(1 << 22) + 8), dict(T=1 << 30),
                dict(T=1 << 31), dict(E=1024, N=1 << 18, K=1 << 18)):
        assert f(lib, **bad) == UNSUPPORTED
    for bad in ("s", "e", "n"):
        assert f(lib, **{bad: None}) == NULL
        assert f(lib, **{bad: A2}) == MISALIGNED


def test_moe_gemm_refusals(lib):
    f = moe_gemm
    assert f(lib, div=3) == SHAPE
    assert f(lib, N=60, tr=1) == SHAPE
    for name in ("X", "W", "Y"):
        assert f(lib, **{name: None}) == NULL
    assert f(lib, X=A4) == f(lib, W=A4) == f(lib, ws=A4) == f(lib, Y=ctypes.c_void_p(0x10001)) == MISALIGNED
    assert f(lib, X=None, W=None, s=None, e=None, n=None, Y=None, T=0) == OK


def test_wgrad_refusals(lib):
    f = wgrad
    for bad in (dict(dd=3), dict(dx=3), dict(N=60), dict(SX=A4, K=72)):
        assert f(lib, **bad) == SHAPE
    for name in ("dY", "X", "dW"):
        assert f(lib, **{name: None}) == NULL
        assert f(lib, **{name: A4}) == MISALIGNED
    assert f(lib, SX=A2) == f(lib, ws=A4) == MISALIGNED
    assert f(lib, T=0, dW=None) == NULL
    # slots past 32-bit byte offsets, which the rows' product takes
    assert f(lib, T=1 << 24, k=16, dd=16, dx=16, N=8, K=8, dY=None) == UNSUPPORTED
    assert f(lib, T=(1 << 24) - 32, k=16, dd=16, dx=16, N=8, K=8, dY=None) == NULL
    assert moe_gemm(lib, T=1 << 24, k=16, div=16, N=8, K=8, X=None) == NULL


def test_rows_out_of_reach(lib):
    """2^34 elements of rows, 2^31 of a checkpoint's scales."""
    big, below = 1 << 14, (1 << 14) - 1
    assert moe_gemm(lib, T=big, k=1, div=1, N=8, K=1 << 20, X=None) == UNSUPPORTED
    assert moe_gemm(lib, T=below, k=1, div=1, N=8, K=1 << 20, X=None) == NULL
    assert moe_gemm(lib, T=1, k=1, div=1, N=1 << 14, K=1 << 20, tr=1, E=1, X=None) == UNSUPPORTED
    assert moe_gemm(lib, T=1, k=1, div=1, N=1 << 14, K=1 << 20, E=1, X=None) == NULL
    for sizes in (dict(N=1 << 20, K=8), dict(N=8, K=1 << 20)):
        assert wgrad(lib, T=big, k=1, dd=1, dx=1, E=1, dY=None, **sizes) == UNSUPPORTED
        assert wgrad(lib, T=below, k=1, dd=1, dx=1, E=1, dY=None, **sizes) == NULL
    tn = lambda M, N, K, SB=None: lib.w4_bf16_gemm_tn(None, A16, SB, A16, M, N, K, None, None)
    assert tn(big, 1 << 20, 8) == tn(big, 8, 1 << 20) == tn((1 << 30) + 1, 8, 8) == UNSUPPORTED
    assert tn(1 << 29, 8, 16, A4) == UNSUPPORTED
    assert tn(below, 1 << 20, 8) == tn(1 << 30, 8, 8) == tn((1 << 29) - 1, 8, 16, A4) == NULL


def test_gemm_tn_refusals(lib):
    f = lambda *a, ws=None: lib.w4_bf16_gemm_tn(*a[:-1], ws, a[-1])
    for M, N, K, SB in ((-1, 8, 8, None), (4, -8, 8, None), (4, 8, -8, None), (4, 12, 8, None), (4, 8, 12, None),
                        (4, 8, 24, A4)):
        assert f(A16, A16, SB, A16, M, N, K, None) == SHAPE
    assert f(None, None, None, None, 4, 0, 8, None) == f(None, None, None, None, 4, 8, 0, None) == OK
    assert f(None, A16, None, A16, 4, 8, 8, None) == NULL
    assert f(A16, None, None, A16, 4, 8, 8, None) == NULL
    assert f(A16, A16, None, None, 4, 8, 8, None) == NULL
    assert f(A4, A16, None, A16, 4, 8, 8, None) == MISALIGNED
    assert f(A16, A4, None, A16, 4, 8, 8, None) == MISALIGNED
    assert f(A16, A16, A2, A16, 4, 16, 16, None) == MISALIGNED
    assert f(A16, A16, None, A4, 4, 8, 8, None) == MISALIGNED
    assert f(A16, A16, None, A16, 4, 8, 8, None, ws=A4) == MISALIGNED
    assert f(A16, A16, None, A16, 1 << 31, 8, 8, None) == UNSUPPORTED
    assert f(A16, A16, None, A16, 4, (1 << 22) + 8, 8, None) == UNSUPPORTED
    assert f(A16, A16, None, A16, 4, 8, (1 << 22) + 8, None) == UNSUPPORTED
    assert f(A16, A16, None, A16, 4, 1 << 21, 1 << 20, None) == UNSUPPORTED


def test_workspaces(lib):
    """Only few results of long sums are split; the parts fill whole results."""
    f, g = lib.w4_bf16_gemm_tn_workspace, lib.w4_bf16_moe_wgrad_workspace
    assert f(8192, 8192, 8192) == f(64, 64, 64) == f(0, 64, 64) == f(64, 0, 64) == 0
    assert f(8192, 64, 64) > 0 and f(8192, 64, 64) % (64 * 64) == 0
    assert f(-1, 8, 8) == f(8, -8, 8) == f(8, 8, (1 << 22) + 8) == f(1 << 31, 8, 8) == -1
    assert g(4096, 8, 64, 4096, 4096) == 0 and g(8192, 1, 1, 64, 64) == f(8192, 64, 64)
    assert g(-1, 1, 1, 8, 8) == g(1, 0, 1, 8, 8) == g(1, 1, 0, 8, 8) == g(1, 1, 1, 0, 8) == -1
    assert g(1 << 24, 17, 1, 8, 8) == g(8, 1, 1025, 8, 8) == g(8, 1, 0x7FFFFFFF, 1 << 22, 1 << 22) == -1
    m = lib.w4_bf16_moe_gemm_workspace
    assert m(8, 1, 1025, 8, 8, 64) == m(8, 1, 1, 8, 8, 1088) == -1
    assert m(4096, 8, 64, 4096, 4096, 256) == m(0, 1, 1, 64, 64, 64) == 0
    assert m(1, 1, 1, 4095, 4096, 64) > 0 and m(1, 1, 1, 4095, 4096, 64) % 4096 == 0
    assert m(-1, 1, 1, 8, 8, 64) == m(1, 1, 1, 8, 8, 32) == m(1 << 30, 2, 1, 8, 8, 64) == -1
    with pytest.raises(ValueError):
        w4.w4_bf16_moe_gemm_workspace(1, 1, 1, 8, 8, 100)
    with pytest.raises(ValueError):
        w4.w4_bf16_gemm_tn_workspace(-1, 8, 8)
    with pytest.raises(ValueError):
        w4.w4_bf16_moe_wgrad_workspace(1, 0, 1, 8, 8)


def test_silu_mul_bwd_refusals(lib):
    f = lib.w4_silu_mul_bwd
    good = [A16, None, A16, None, 4, 64, A16, A16, A4, None]

    def call(**at):
        a = list(good)
        for i, v in at.items():
            a[int(i[1:])] = v
        return f(*a)
    assert call(a4=-1) == call(a5=-8) == call(a5=12) == SHAPE
    assert call(a4=1 << 31) == call(a5=(1 << 22) + 8) == UNSUPPORTED
    assert call(a0=None) == call(a2=None) == call(a6=None) == NULL
    assert call(a0=A4) == call(a1=A2) == call(a2=A4) == call(a3=A2) == call(a6=A4) == call(a7=A4) == MISALIGNED
    assert call(a8=A2) == MISALIGNED
    assert f(None, None, None, None, 0, 64, None, None, None, None) == OK
    assert f(None, None, None, None, 4, 0, None, None, None, None) == OK


def test_binding_refuses_cpu_tensors_and_types():
    x = torch.zeros((8, 64), dtype=torch.bfloat16)
    ids = torch.zeros((4, 2), dtype=torch.int32)
    i = torch.zeros(1024, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        w4.w4_bf16_moe_gemm(x, x.view(1, 8, 64), i, i, i, 4, 2, 64, 1)
    with pytest.raises(ValueError, match="GPU"):
        w4.w4_bf16_moe_wgrad(x, x, i, i, i, 1, 4, 2, 64, 1, 1)
    with pytest.raises(ValueError, match="GPU"):
        w4.w4_bf16_gemm_tn(x, x)
    with pytest.raises(ValueError, match="GPU"):
        w4.w4_silu_mul_bwd(x, x)
    with pytest.raises(TypeError):
        w4.w4_bf16_gemm_tn(x.float(), x)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_train(x[:4], ids, torch.zeros((4, 2)), x.view(1, 8, 64), x.view(1, 64, 8))
