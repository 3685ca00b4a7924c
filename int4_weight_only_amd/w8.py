"""Training with 8-bit floating-point products: a linear layer whose forward
and input gradient run on e4m3 codes with block scales, with a
straight-through estimator ("INT4 QAT end-to-end for RL" §2.1 for the
estimator; the W8A8-FP8 rollout it is compared with is the product here).

Forward: Y = Q_rows(X) * Q_blocks(W)^T (``w8_quantize_rows``,
``w8_quantize_blocks``, ``w8a8_gemm``).  Backward: the rounding counts as the
identity, so
  dX = Q_rows(dY) * Q_blocks(W)     ``w8a8_gemm`` on the transposed codes: a
                                    128 x 128 block transposes onto itself, so
                                    they are the forward's numbers, written by
                                    the same call
  dW = dY^T * X                     bf16, unquantized operands
                                    (``w4_bf16_transpose``, ``w4_bf16_gemm_nt``)
which covers fewer than 2^22 tokens: more of them are refused in the forward
where W needs a gradient.  The master weight stays bf16.  The backward is not
differentiable again.  To capture a backward into a graph, take gradients with
``torch.autograd.grad``, or let no eager graph of the same leaves be alive.
"""

import torch
from torch.autograd.function import once_differentiable

from . import (w4_bf16_gemm_nt, w4_bf16_transpose, w8_quantize_blocks, w8_quantize_rows, w8a8_gemm)

__all__ = ["W8Linear", "w8_linear"]


def _padded(rows):
    """Columns of the weight gradient's transposed operands: whole 128-byte
    lines, their ends zero (the product of [4096, 2056] and [5120, 2056] takes
    109 us, 97 in 2112)."""
    return (rows + 63) // 64 * 64


class W8Linear(torch.autograd.Function):
    """y = Q(x) * Q(W)^T with a straight-through backward."""

    @staticmethod
    def forward(ctx, X, W, grad=True):
        N, K = W.shape
        if X.shape[-1] != K:
            raise ValueError(f"X has {X.shape[-1]} features, W expects {K}")
        W = W.contiguous()
        X2 = X.reshape(-1, K).contiguous()
        # needs_input_grad goes by the inputs alone, also under torch.no_grad()
        need_dx, need_dw = (n and grad for n in ctx.needs_input_grad[:2])
        if need_dx and N % 16:
            raise ValueError(f"the W8A8 input gradient needs N % 16 == 0 (N = {N})")
        if need_dw and min(256, max(N, K)) * _padded(X2.shape[0]) * 2 >= 1 << 31:
            raise ValueError(f"the W8A8 weight gradient covers fewer than 2^22 tokens, got {X2.shape[0]}")
        W8, SW, WT8, ST = w8_quantize_blocks(W, transposed=need_dx)
        Y = w8a8_gemm(*w8_quantize_rows(X2), W8, SW)
        ctx.save_for_backward(X2 if need_dw else None, WT8, ST)
        ctx.x_shape, ctx.n = X.shape, N
        return Y.reshape(*X.shape[:-1], N)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        X2, WT8, ST = ctx.saved_tensors
        dY = grad_out.reshape(-1, ctx.n).to(torch.bfloat16).contiguous()
        dX = dW = None
        if ctx.needs_input_grad[0]:
            dX = w8a8_gemm(*w8_quantize_rows(dY), WT8, ST).reshape(ctx.x_shape)
        if ctx.needs_input_grad[1]:
            rows = _padded(dY.shape[0])
            dW = w4_bf16_gemm_nt(w4_bf16_transpose(dY, rows), w4_bf16_transpose(X2, rows))
        return dX, dW, None


def w8_linear(X, W):
    """Linear layer without bias on e4m3 operands: X bf16 [..., K], W bf16
    [N, K] (K % 16 == 0, and N % 16 == 0 where X needs a gradient) -> bf16
    [..., N]."""
    return W8Linear.apply(X, W, torch.is_grad_enabled())
