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

pytestmark = pytest.mark.gpu


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
