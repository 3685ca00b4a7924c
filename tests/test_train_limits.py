"""What the training layers refuse in the forward since their backward could not compute
it.  Sizes only: no GPU."""

import pytest
import torch

import int4_weight_only_amd as w4
from int4_weight_only_amd import moe


def moe_sizes(T=32, k=4, E=8, H=128, I=64, B=64, checkpoint=False, x=True, w=True, up=True, dn=True):
    return moe.check_moe_backward(T, k, E, H, I, B, checkpoint, x, w, up, dn)


@pytest.mark.parametrize("checkpoint", [False, True])
def test_moe_train_sizes(checkpoint):
    for good in (dict(), dict(B=1024), dict(B=192), dict(T=0), dict(T=1, k=1, E=1, H=16, I=8),
                 dict(T=4096, k=8, E=384, H=7168, I=2048, B=128)):
        moe_sizes(checkpoint=checkpoint, **good)
    for bad in (dict(B=16), dict(B=32), dict(B=96), dict(B=1088), dict(B=16, T=0), dict(E=1025)):
        with pytest.raises(ValueError):
            moe_sizes(checkpoint=checkpoint, **bad)


def test_moe_train_limits_of_each_gradient():
    """The weight gradients take 2^28 slots, the products more; rows of 2^34 elements nothing."""
    slots = dict(T=1 << 25, k=8, E=1, H=32, I=16)
    for want in (dict(up=False), dict(dn=False)):
        with pytest.raises(ValueError, match="weight gradient"):
            moe_sizes(**slots, **want)
    moe_sizes(**slots, up=False, dn=False)
    moe_sizes(**{**slots, "T": (1 << 25) - 8})
    rows = dict(T=1 << 20, k=16, E=1, H=64, I=512)            # dH1: 2^24 rows of 1024
    with pytest.raises(ValueError, match="product"):
        moe_sizes(**rows, up=False, dn=False)
    moe_sizes(**rows, x=False, up=False)


class Huge:
    """A bf16 matrix of M rows, as far as the linear layers' checks look at it."""

    def __init__(self, M, K):
        self.shape = (M, K)

    def reshape(self, *shape):
        return self

    def contiguous(self):
        return self


class Context:
    needs_input_grad = (True, True, False, False)


@pytest.mark.parametrize("M,K", [((1 << 30) + 16, 64), (1 << 29, 32), (1 << 24, 1024)])
def test_linear_checkpoint_limits(M, K, monkeypatch):
    """Rows, scales and elements past what the product from codes takes, before anything runs."""
    from int4_weight_only_amd import qat, w8

    def ran(*a, **k):
        raise AssertionError("a kernel before the refusal")
    for module, names in ((w8, ("w8_quantize_blocks", "w8_quantize_rows", "w8a8_gemm")),
                          (qat, ("w4_quantize_pack", "w8_quantize_rows", "w4a16_gemm"))):
        for n in names:
            monkeypatch.setattr(module, n, ran)
    with pytest.raises(ValueError, match="from a checkpoint"):
        w8.W8Linear.forward(Context(), Huge(M, K), Huge(64, K), True, True)
    with pytest.raises(ValueError, match="from a checkpoint"):
        qat.Int4QATLinear.forward(Context(), Huge(M, K), Huge(64, K), True, True)


def test_linear_checkpoint_sizes_that_are_taken():
    """dY and the codes: fewer than 2^34 elements each."""
    for M, N, K in ((0, 16, 32), (1, 8, 16), ((1 << 22) - 1, 4096, 4080), ((1 << 29) - 1, 8, 16)):
        w4.check_checkpoint_wgrad(M, N, K)
    with pytest.raises(ValueError):
        w4.check_checkpoint_wgrad(1 << 22, 4096, 4080)


def test_no_pairs_per_token_is_refused_as_an_argument():
    """k = 0 with its divisor: not a division by zero."""
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="meta")
    i = torch.zeros(64, dtype=torch.int32, device="meta")
    for T, k in ((4, 0), (-1, 1)):
        with pytest.raises(ValueError, match="T or k"):
            w4.w4_bf16_moe_gemm(x, x.view(1, 0, 64), i, i, i, T, k, 64, k)
        with pytest.raises(ValueError, match="T or k"):
            w4.w4_bf16_moe_wgrad(x, x, i, i, i, 1, T, k, 64, k, 1)


def test_moe_train_checks_what_a_gradient_runs():
    """Weights of 2^34 elements an expert, which the input gradient's product refuses: the down
    weights' own gradient does not run it."""
    big = dict(T=8, k=1, E=1, H=1 << 17, I=1 << 17)
    moe_sizes(**big, x=False, w=False, up=False)
    for only in ("x", "w", "up"):
        with pytest.raises(ValueError, match="product"):
            moe_sizes(**big, **{n: n == only for n in ("x", "w", "up", "dn")})
