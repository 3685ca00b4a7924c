"""The scored router against the fp64 oracle.

Indices are equal: both sides hold choice values in 64 bits.  Weights and
gradients are 64-bit values rounded to fp32 once, 2^-24 of the value; 2^-23
leaves room for the 64-bit roundings and the fp32 rounding of `scale`.
"""

import numpy as np
import pytest
import torch

import int4_weight_only_amd as w4
from int4_weight_only_amd import moe
import synth
from gpu_util import dev, down, say, up
from oracle import w8 as ow8

pytestmark = pytest.mark.gpu

RULES = [dict(), dict(renorm=False, scale=0.5), dict(sigmoid=True), dict(sigmoid=True, renorm=False),
         dict(sigmoid=True, bias=True, scale=2.5), dict(bias=True, groups=4, topk_groups=2),
         dict(sigmoid=True, bias=True, groups=4, topk_groups=2, group_top=2),
         dict(groups=2, topk_groups=1, group_top=2, renorm=False)]


def check(lg, k, rule, seed=0):
    rule = dict(rule)
    E = lg.shape[1]
    if rule.get("bias") is True:
        rule["bias"] = np.random.default_rng(seed).normal(size=E).astype(np.float32) * 0.1
    on_gpu = dict(rule, bias=up(rule["bias"])) if "bias" in rule else rule
    ids, w = w4.w4_moe_route_scored(up(lg), k, **on_gpu)
    ids_ref, w_ref = ow8.route_scored(lg, k, **rule)
    np.testing.assert_array_equal(down(ids), ids_ref)
    np.testing.assert_allclose(down(w), w_ref, rtol=2.0 ** -23, atol=1e-45)
    dw = np.random.default_rng(seed + 1).normal(size=w_ref.shape).astype(np.float32)
    how = {n: rule[n] for n in ("sigmoid", "renorm", "scale") if n in rule}
    got = down(w4.w4_moe_route_scored_bwd(up(lg), ids, w, up(dw), **how)).astype(np.float64)
    ref = ow8.route_scored_grad(lg, ids_ref, down(w), dw, **how)
    # a gradient is a difference of terms of the size of scale |dw|: 64-bit
    # roundings of those, and one fp32 rounding
    size = 2.5 * np.abs(dw).max() if dw.size else 1.0
    assert np.all(np.abs(got - ref) <= 2.0 ** -23 * np.abs(ref) + 2.0 ** -45 * size + 1e-45)
    return down(ids), down(w)


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("T,E,k", [(1, 16, 4), (7, 64, 8), (33, 128, 8), (5, 384, 8), (3, 1024, 16), (9, 200, 3), (4, 8, 4),
                                   (2, 512, 1), (6, 260, 16)])
def test_route(rule, T, E, k):
    say(f"route_scored T={T} E={E} k={k} {rule}")
    check(synth.router_logits(T, E, 3).numpy(), k, rule)


@pytest.mark.parametrize("rule", RULES)
def test_masks_infinities_and_ties(rule):
    E, k = 16, 6
    lg = np.random.default_rng(1).normal(size=(9, E)).astype(np.float32)
    lg[0, :] = -np.inf
    lg[1, :] = np.nan
    lg[2, 3:] = -np.inf                          # fewer experts than picks
    lg[3, :] = 0                                 # all equal
    lg[4, ::2] = np.finfo(np.float32).min        # a mask of the lowest value
    lg[5, 4] = np.inf
    lg[6, [1, 9]] = np.inf
    lg[7, :] = np.linspace(-300, 300, E, dtype=np.float32)
    lg[8, [2, 5, 11]] = lg[8, 0] + 4             # equal and largest
    say(f"route_scored masks {rule}")
    if rule.get("bias") and rule.get("groups", 1) == 1:
        rule = dict(rule, bias=np.where(np.arange(E) == 7, -np.inf, 0.01 * np.arange(E)).astype(np.float32))
    if rule.get("groups", 1) > 1:
        k = 4
    ids, w = check(lg, k, rule)
    for t in (0, 1):
        assert list(ids[t]) == list(range(k)) and not w[t].any()
    assert all(len(set(r)) == k for r in ids)


@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("groups,topk_groups", [(1, 1), (4, 2)])
@pytest.mark.parametrize("E", [16, 256])
def test_scores_that_vanish_in_64_bits(E, groups, topk_groups, tied):
    # the bias picks experts whose softmax is zero, or nearly, beside one logit:
    # the same weights whether their choice values are apart or equal
    lg = np.zeros((7, E), np.float32)
    lg[:, 9] = [1000, 800, 700, 650, 590, 300, np.inf]
    lg[:6, 3] = [0, 0, -5, 1, 2, -400]
    bias = np.zeros(E, np.float32)
    bias[[1, 3]] = [3.0, 3.0 if tied else 2.5]
    rule = dict(groups=groups, topk_groups=topk_groups)
    say(f"route_scored vanishing scores E={E} groups={groups} tied={tied}")
    ids, w = w4.w4_moe_route_scored(up(lg), 2, bias=up(bias), **rule)
    ids_ref, p = ow8.route_scored(lg, 2, bias=bias, **rule)
    np.testing.assert_array_equal(down(ids), ids_ref)
    assert np.all(ids_ref == [1, 3]) and not p[[0, 1, 6]].any() and p[2:6].any(1).all()
    np.testing.assert_allclose(down(w), p, rtol=2.0 ** -23, atol=1e-45)
    # the gradient by its formula: the oracle's divides by the square of a sum
    # that is zero in 64 bits
    dw = np.random.default_rng(8).normal(size=p.shape).astype(np.float32)
    ref = np.zeros(lg.shape)
    np.put_along_axis(ref, ids_ref.astype(np.int64), p * (dw - (p * dw).sum(1, keepdims=True)), 1)
    got = down(w4.w4_moe_route_scored_bwd(up(lg), ids, w, up(dw))).astype(np.float64)
    assert np.all(np.abs(got - ref) <= 2.0 ** -23 * np.abs(ref) + 2.0 ** -45 * np.abs(dw).max())


@pytest.mark.parametrize("E,k,groups,topk_groups", [(64, 4, 8, 3), (128, 8, 8, 4), (256, 8, 32, 3), (384, 6, 64, 2), (512, 16, 2, 1),
                                                    (1024, 5, 16, 5), (24, 4, 3, 2), (384, 8, 6, 3), (64, 2, 64, 5), (90, 6, 10, 4)])
@pytest.mark.parametrize("sigmoid,group_top", [(True, 2), (False, 1)])
def test_groups_in_every_layout(E, k, groups, topk_groups, sigmoid, group_top):
    # a group in neighbouring lanes' registers or in LDS, with masked experts,
    # masked groups, equal groups and rows of few experts
    rule = dict(sigmoid=sigmoid, groups=groups, topk_groups=topk_groups, group_top=group_top, bias=True)
    say(f"route_scored groups E={E} k={k} {rule}")
    lg = synth.router_logits(12, E, 6).numpy().copy()
    per = E // groups
    lg[1, :per] = -np.inf
    lg[2, per:] = -np.inf
    lg[3, ::2] = np.nan
    lg[4] = 0
    lg[5, :] = np.tile(lg[5, :per], groups)
    lg[6, 1:] = -np.inf
    lg[7, E - per:] += 50
    lg[8, :] = -np.inf
    lg[9, E - 1] = np.inf
    check(lg, k, rule)
    check(lg, k, dict(rule, bias=np.zeros(E, np.float32)))
    assert topk_groups * per >= k


def test_many_rows_with_groups_agree_with_64_bits():
    T, E, k, groups, kept = 20000, 256, 8, 8, 4
    lg = torch.randn(T, E, generator=torch.Generator().manual_seed(4)).to(dev())
    b = (torch.randn(E, generator=torch.Generator().manual_seed(5)) * 0.05).to(dev())
    say("route_scored many rows with groups")
    ids, _ = w4.w4_moe_route_scored(lg, k, sigmoid=True, bias=b, groups=groups, topk_groups=kept, group_top=2)
    c = (torch.sigmoid(lg.double()) + b.double()).view(T, groups, E // groups)
    worth = torch.sort(c, dim=2, descending=True).values[:, :, :2].sum(2)
    best = torch.sort(worth, dim=1, descending=True, stable=True).indices[:, :kept]
    keep = torch.zeros(T, groups, dtype=torch.bool, device=dev()).scatter_(1, best, True)
    c = torch.where(keep[:, :, None], c, -torch.inf).view(T, E)
    ref = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids.long(), ref)


def test_refuses_second_derivatives():
    x = synth.router_logits(3, 16, 7).to(dev()).requires_grad_()
    say("route_scored second derivative")
    g, = torch.autograd.grad(moe.route_scored(x, 2)[1].square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_single_expert_and_empty():
    say("route_scored E=1")
    ids, w = w4.w4_moe_route_scored(torch.zeros(3, 1, device=dev()), 1, sigmoid=True, renorm=False)
    assert not ids.any() and (w == 0.5).all()
    ids, w = w4.w4_moe_route_scored(torch.zeros(0, 8, device=dev()), 2)
    assert ids.shape == w.shape == (0, 2)


def test_many_rows_agree_with_64_bits():
    # near ties: 20000 rows, sigmoid + bias, checked against torch in fp64
    T, E, k = 20000, 384, 8
    lg = torch.randn(T, E, generator=torch.Generator().manual_seed(2)).to(dev())
    b = (torch.randn(E, generator=torch.Generator().manual_seed(3)) * 0.05).to(dev())
    say("route_scored many rows")
    ids, _ = w4.w4_moe_route_scored(lg, k, sigmoid=True, bias=b)
    c = torch.sigmoid(lg.double()) + b.double()
    ref = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids.long(), ref)


def test_backward_repeated_and_foreign_ids():
    lg = synth.router_logits(4, 12, 5).numpy()
    ids = np.array([[3, 3, 5], [0, 11, 0], [-1, 2, 12], [7, 7, 7]], np.int32)
    w = np.ones((4, 3), np.float32)
    w[1, 1] = 0
    dw = np.random.default_rng(7).normal(size=(4, 3)).astype(np.float32)
    for how in (dict(renorm=False), dict(sigmoid=True, renorm=False), dict(renorm=True), dict(sigmoid=True)):
        say(f"route_scored_bwd ids {how}")
        got = down(w4.w4_moe_route_scored_bwd(up(lg), up(ids), up(w), up(dw), **how))
        ref = ow8.route_scored_grad(lg, ids, w, dw, **how)
        np.testing.assert_allclose(got, ref, rtol=2.0 ** -22, atol=2.0 ** -45)


@pytest.mark.parametrize("rule", [dict(sigmoid=True, groups=2, topk_groups=1, group_top=2, scale=2.0), dict(renorm=False), dict()])
def test_autograd_against_differences(rule):
    T, E, k = 3, 12, 3
    lg = synth.router_logits(T, E, 9)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(1))
    x = lg.to(dev()).requires_grad_()
    say(f"route_scored autograd {rule}")
    ids, w = moe.route_scored(x, k, **rule)
    assert not ids.requires_grad
    (w * dw.to(dev())).sum().backward()
    ids, h = down(ids), 1e-5

    def loss(v):
        s = np.stack([ow8.scores(r, rule.get("sigmoid", False)) for r in v])
        p = np.take_along_axis(s, ids, 1)
        p = p / p.sum(1, keepdims=True) if rule.get("renorm", True) else p
        return (rule.get("scale", 1.0) * p * dw.numpy()).sum()
    v = lg.numpy().astype(np.float64)
    for t in range(T):
        for e in range(E):
            d = np.zeros_like(v)
            d[t, e] = h
            # central differences: h^2 of the third derivative, and fp32's own rounding of the gradient
            assert abs((loss(v + d) - loss(v - d)) / (2 * h) - float(x.grad[t, e])) < 1e-6


def test_graph_replay_forward_and_backward():
    T, E, k = 40, 64, 4
    how = dict(sigmoid=True, scale=1.5)
    lg, dw = synth.router_logits(T, E, 1, device=dev()), torch.ones(T, k, device=dev())
    ids, w = torch.empty(T, k, dtype=torch.int32, device=dev()), torch.empty(T, k, device=dev())
    dl = torch.empty(T, E, device=dev())

    def call():
        w4.w4_moe_route_scored(lg, k, groups=4, topk_groups=2, group_top=2, topk_ids=ids, topk_weights=w, **how)
        w4.w4_moe_route_scored_bwd(lg, ids, w, dw, grad_logits=dl, **how)
    say("route_scored graph")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for r in range(4):
        lg.copy_(synth.router_logits(T, E, 10 + r, device=dev()))
        dw.copy_(synth.router_logits(T, k, 20 + r, device=dev()))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (ids, w, dl)]
        call()
        for a, b in zip(got, (ids, w, dl)):
            assert torch.equal(a, b), f"replay {r}"
