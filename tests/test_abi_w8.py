"""The W8A8 and scored-router entry points without a GPU: sizes, refusals of
the C ABI (nothing here reaches the HIP runtime), and of the binding."""

import ctypes

import pytest
import torch

import int4_weight_only_amd as w4
from int4_weight_only_amd import _lib, moe, w8

A16, A4, A2, A1 = (ctypes.c_void_p(0x10000 + o) for o in (0, 4, 2, 1))
OK, NULL, SHAPE, MISALIGNED, UNSUPPORTED = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_scale_cols(lib):
    assert [lib.w8_scale_cols(k) for k in (0, 16, 512, 528, 4096)] == [0, 4, 4, 8, 32]
    assert lib.w8_scale_cols(-1) == -1
    with pytest.raises(ValueError):
        w4.w8_scale_cols(-1)


def test_pick_block_size(lib):
    for T, k, E, B in ((1, 1, 1, 16), (256, 8, 128, 64), (2048, 8, 32, 256), (0, 8, 4, 16), (64, 8, 64, 16),
                       (65, 8, 64, 64), (43, 1, 1, 128), (42, 1, 1, 64), (85, 1, 1, 128), (86, 1, 1, 256),
                       (1 << 50, 8, 64, 256)):
        assert lib.w8_pick_block_size(T, k, E) == B
    assert lib.w8_pick_block_size(-1, 1, 1) == lib.w8_pick_block_size(1, 0, 1) == 0
    assert lib.w8_pick_block_size(1, 1, 0) == 0


def test_quantize_rows_refusals(lib):
    f = lib.w8_quantize_rows
    assert f(A16, 4, 24, A16, A4, None) == SHAPE
    assert f(A16, -1, 32, A16, A4, None) == SHAPE
    assert f(None, 0, 32, None, None, None) == OK
    assert f(None, 4, 0, None, None, None) == OK
    assert f(None, 4, 32, A16, A4, None) == NULL
    assert f(A16, 4, 32, None, A4, None) == NULL
    assert f(A16, 4, 32, A16, None, None) == NULL
    assert f(A4, 4, 32, A16, A4, None) == MISALIGNED
    assert f(A16, 4, 32, A4, A4, None) == MISALIGNED
    assert f(A16, 4, 32, A16, A2, None) == MISALIGNED
    assert f(A16, 4, (1 << 22) + 16, A16, A4, None) == UNSUPPORTED
    assert f(A16, 1 << 31, 16, A16, A4, None) == UNSUPPORTED


def test_silu_mul_quantize_refusals(lib):
    f = lib.w8_silu_mul_quantize
    assert f(A16, 4, 24, A16, A4, None) == SHAPE
    assert f(None, 0, 32, None, None, None) == OK
    assert f(None, 4, 32, A16, A4, None) == NULL
    assert f(A16, 4, 32, A16, A2, None) == MISALIGNED


def test_quantize_blocks_refusals(lib):
    f = lib.w8_quantize_blocks
    assert f(A16, 4, 24, A16, A4, None, None, None) == SHAPE
    assert f(A16, 24, 32, A16, A4, A16, A4, None) == SHAPE      # transposed: N % 16
    assert f(None, 0, 32, None, None, None, None, None) == OK
    assert f(A16, 32, 32, A16, A4, A16, None, None) == NULL
    assert f(A16, 32, 32, A16, A4, None, A4, None) == NULL
    assert f(A16, 32, 32, None, A4, None, None, None) == NULL
    assert f(A16, 32, 32, A16, A4, A4, A4, None) == MISALIGNED
    assert f(A16, 32, 32, A16, A4, A16, A2, None) == MISALIGNED
    assert f(A16, 1 << 31, 16, A16, A4, None, None, None) == UNSUPPORTED


def test_gemm_refusals(lib):
    f = lib.w8a8_gemm
    assert f(A16, A4, A16, A4, A2, -1, 16, 32, None) == SHAPE
    assert f(A16, A4, A16, A4, A2, 4, 16, 40, None) == SHAPE
    assert f(None, None, None, None, None, 0, 16, 32, None) == OK
    assert f(None, None, None, None, None, 4, 0, 32, None) == OK
    assert f(A16, A4, A16, A4, None, 4, 16, 32, None) == NULL
    assert f(A16, None, A16, A4, A2, 4, 16, 32, None) == NULL
    assert f(A16, A4, A16, A4, A1, 4, 16, 32, None) == MISALIGNED
    assert f(A16, A4, A4, A4, A2, 4, 16, 32, None) == MISALIGNED
    assert f(A16, A2, A16, A4, A2, 4, 16, 32, None) == MISALIGNED
    assert f(A16, A4, A16, A4, A2, 4, 16, (1 << 22) + 16, None) == UNSUPPORTED
    assert f(A16, A4, A16, A4, A2, 1 << 24, 1 << 24, 16, None) == UNSUPPORTED


def test_moe_gemm_refusals(lib):
    def f(T=4, k=2, E=3, N=16, K=32, B=16, div=2, X=A16, S=A4, W=A16, ids=A4, Y=A2):
        return lib.w8a8_moe_gemm(X, S, W, S, ids, A4, A4, Y, T, k, E, N, K, B, div, None)
    assert f(T=-1) == f(k=0) == f(E=0) == f(N=0) == f(K=24) == f(K=0) == SHAPE
    assert f(B=8) == f(B=24) == f(B=0) == f(div=3) == SHAPE
    assert f(T=0, X=None) == OK
    assert f(B=1040) == f(E=1025) == f(K=(1 << 22) + 16) == f(T=1 << 31) == UNSUPPORTED
    assert f(N=1 << 30, K=1 << 20) == UNSUPPORTED
    assert f(X=None) == f(S=None) == f(ids=None) == f(Y=None) == NULL
    assert f(X=A4) == f(W=A4) == f(S=A2) == f(ids=A2) == f(Y=A1) == MISALIGNED


def test_moe_gemm_swiglu_refusals(lib):
    def f(T=4, k=2, E=3, I=128, K=32, B=256, div=2, X=A16, S=A4, A=A16, SA=A4):
        return lib.w8a8_moe_gemm_swiglu(X, S, A16, S, A4, A4, A4, A, SA, T, k, E, I, K, B, div, None)
    assert f(I=0) == f(I=24) == f(T=-1) == f(K=24) == f(B=8) == f(div=3) == SHAPE
    assert f(I=144) == f(B=64) == f(B=320) == f(I=1 << 31, X=None) == f(T=1 << 26, K=1024) == UNSUPPORTED
    assert f(T=0, X=None) == OK
    assert f(X=None) == f(A=None) == f(SA=None) == NULL
    assert f(X=A4) == f(A=A4) == f(SA=A2) == MISALIGNED


def test_route_scored_refusals(lib):
    def f(T=4, E=16, k=2, groups=1, tg=1, top=1, lg=A4, bias=None, ids=A4, w=A4):
        return lib.w4_moe_route_scored(lg, bias, T, E, k, 1, groups, tg, top, 1, 1.0, ids, w, None)
    assert f(T=-1) == f(E=0) == f(k=0) == f(groups=3) == f(groups=0) == f(top=3) == f(top=0) == SHAPE
    assert f(groups=4, tg=5) == f(tg=0) == SHAPE
    assert f(k=17, E=32) == f(k=5, E=4) == f(E=1040) == UNSUPPORTED
    assert f(groups=8, tg=1, k=3) == f(E=130, groups=65, tg=65) == UNSUPPORTED
    assert f(T=(1 << 25) + 1) == UNSUPPORTED
    assert f(T=0, lg=None) == OK
    assert f(lg=None) == f(ids=None) == f(w=None) == NULL
    assert f(lg=A2) == f(bias=A2) == f(ids=A2) == f(w=A2) == MISALIGNED


def test_route_scored_bwd_refusals(lib):
    def f(T=4, E=16, k=2, lg=A4, ids=A4, w=A4, g=A4, out=A4):
        return lib.w4_moe_route_scored_bwd(lg, ids, w, g, T, E, k, 1, 1, 1.0, out, None)
    assert f(T=-1) == f(E=0) == f(k=0) == SHAPE
    assert f(k=17, E=32) == f(E=1040) == f(T=(1 << 25) + 1) == UNSUPPORTED
    assert f(T=0, lg=None) == OK
    assert f(lg=None) == f(ids=None) == f(w=None) == f(g=None) == f(out=None) == NULL
    assert f(lg=A2) == f(out=A2) == MISALIGNED


def test_binding_refuses_cpu_tensors_and_wrong_types():
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    q, s = x.to(torch.float8_e4m3fn), torch.zeros(4, 4, dtype=torch.uint8)
    for call in (lambda: w4.w8_quantize_rows(x), lambda: w4.w8_quantize_blocks(x),
                 lambda: w4.w8_silu_mul_quantize(x), lambda: w8.w8_linear(x, x),
                 lambda: w4.w8a8_gemm(q, s, q, s),
                 lambda: w4.w8a8_moe_gemm(q, s, q[None], s, s, s, s, 4, 1, 16, 1),
                 lambda: w4.w4_moe_route_scored(torch.zeros(2, 4), 2),
                 lambda: moe.route_scored(torch.zeros(2, 4), 2)):
        with pytest.raises(ValueError, match="on a GPU"):
            call()
    for call in (lambda: w4.w8_quantize_rows(x.float()), lambda: w4.w8a8_gemm(x, s, q, s),
                 lambda: w4.w4_moe_route_scored(x, 2)):
        with pytest.raises(TypeError):
            call()


def test_weight_gradient_limits(lib):
    f = lib.w4_bf16_gemm_nt
    K = 1 << 22
    assert f(None, None, A2, 16384, 8192, 70016, None) == NULL      # operands past 2 GiB: covered
    assert f(None, None, A2, 1 << 20, 256, K - 8, None) == NULL
    assert f(None, None, A2, 255, 100, K, None) == NULL
    assert f(None, None, A2, 256, 100, K, None) == f(None, None, A2, 100, 256, K, None) == UNSUPPORTED
    assert f(None, None, A2, 1, 1, 1 << 30, None) == UNSUPPORTED
    x, w = torch.zeros(1, 16, dtype=torch.bfloat16).expand(K, 16), torch.zeros(256, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="tokens"):
        w8.w8_linear(x, w.requires_grad_())


def test_launch_limit_counts_the_launch(lib):
    def moe(B, T=1 << 17, k=8, N=8192, E=16, K=64):
        return lib.w8a8_moe_gemm(None, A4, A16, A4, A4, A4, A4, A2, T, k, E, N, K, B, k, None)
    # 2^20 pairs x 8192: tiles of 64 rows and more start far fewer than 2^32 threads, those of 16 do not
    assert moe(256) == moe(128) == moe(64) == NULL
    assert moe(16) == UNSUPPORTED
    assert moe(32) == NULL and moe(32, N=16384) == UNSUPPORTED
    f = lib.w8a8_moe_gemm_swiglu
    assert f(None, A4, A16, A4, A4, A4, A4, A16, A4, 1 << 17, 8, 16, 8192, 64, 256, 8, None) == NULL
    assert lib.w8a8_gemm(None, A4, A16, A4, A2, 1, 100000000, 16, None) == NULL
    assert lib.w8a8_gemm(None, A4, A16, A4, A2, 1, 1 << 27, 16, None) == UNSUPPORTED


def test_expert_layer_refuses_inputs_that_want_gradients():
    x, lg, w = torch.zeros(2, 32, dtype=torch.bfloat16), torch.zeros(2, 4), torch.zeros(2, 1)
    ids = torch.zeros(2, 1, dtype=torch.int32)
    e = moe.ExpertWeightsW8(torch.zeros(4, 32, 32, dtype=torch.bfloat16).to(torch.float8_e4m3fn), torch.zeros(4, 1, 4))
    for call in (lambda: moe.moe_layer_w8(x.clone().requires_grad_(), lg, 1, e, e),
                 lambda: moe.moe_layer_w8(x, lg.clone().requires_grad_(), 1, e, e),
                 lambda: moe.moe_forward_w8(x.clone().requires_grad_(), ids, w, e, e),
                 lambda: moe.moe_forward_w8(x, ids, w.clone().requires_grad_(), e, e)):
        with pytest.raises(ValueError, match="no backward"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="on a GPU|do not match"):
            call()


def test_linear_without_gradients_has_no_limits_of_theirs():
    x = torch.zeros(2, 16, dtype=torch.bfloat16, requires_grad=True)
    w = torch.zeros(24, 16, dtype=torch.bfloat16, requires_grad=True)
    many = torch.zeros(1, 16, dtype=torch.bfloat16).expand(1 << 22, 16)
    with pytest.raises(ValueError, match="N % 16"):
        w8.w8_linear(x, w)
    with torch.no_grad():
        for a, b in ((x, w), (many, torch.zeros(256, 16, dtype=torch.bfloat16, requires_grad=True))):
            with pytest.raises(ValueError, match="on a GPU"):
                w8.w8_linear(a, b)
