"""Pins of the FP8 oracle: the formats' closed forms, torch's own e4m3 cast
on the CPU, the scale rule's two inequalities, and the router against brute
force and difference quotients."""

import itertools

import numpy as np
import pytest
import torch

import synth
from oracle import bf16, w8


def test_e4m3_closed_forms():
    v = w8.e4m3_values(np.arange(256, dtype=np.uint8))
    assert v[0x7E] == 448 and v[0xFE] == -448 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6
    assert np.isnan(v[0x7F]) and np.isnan(v[0xFF]) and v[0x38] == 1.0
    assert np.all(np.diff(v[:127]) > 0)
    np.testing.assert_array_equal(w8.e4m3_codes(v[:127]), np.arange(127))


def test_e4m3_rounding_matches_torch():
    mid = (w8._POSITIVE[1:] + w8._POSITIVE[:-1]) / 2          # every tie
    x = np.concatenate([mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9),
                        np.random.default_rng(0).uniform(-448, 448, 5000)]).astype(np.float32)
    x = np.concatenate([x, -x])
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(w8.e4m3_codes(x), ref)


@pytest.mark.parametrize("amax", [448.0, 448.0000001, 1.75, 1.7500001, 1.0, 2.0 ** -126, 2.0 ** -133, 3.3e38,
                                  448 * 2.0 ** -127])
def test_scale_is_the_smallest_that_fits(amax):
    e = w8.exponent(amax)
    assert amax <= 448 * 2.0 ** e and e >= -127
    assert e == -127 or amax > 448 * 2.0 ** (e - 1)
    assert w8.exponent(0.0) == 0


def test_quantize_error_bound_and_layout():
    b = synth.bits(synth.activations(3, 656, 1))
    q, s = w8.quantize_rows(b)
    assert s.shape == (3, 8) and np.all(s[:, 6:] == 127)
    x, y = bf16.to_f32(b).astype(np.float64), w8.dequant(q, s, 1)
    step = np.repeat(2.0 ** (s.astype(float) - 127), 128, 1)[:, :656]
    assert np.all(np.abs(x - y) <= np.maximum(np.abs(x) * 2.0 ** -4, step * 2.0 ** -10))


def test_square_blocks_transpose_onto_themselves():
    b = synth.bits(synth.weights(272, 400, 2))
    q, s = w8.quantize_blocks(b)
    qt, st = w8.quantize_blocks(np.ascontiguousarray(b.T))
    np.testing.assert_array_equal(qt, q.T)
    np.testing.assert_array_equal(st[:4, :3], s[:3, :4].T)


def test_bad_blocks_are_nan():
    b = synth.bits(synth.activations(2, 256, 3)).copy()
    b[0, 5], b[1, 200] = 0x7F80, 0x7FC1
    q, s = w8.quantize_rows(b)
    assert s[0, 0] == s[1, 1] == 255 and np.all(q[0, :128] == 0x7F) and s[0, 1] != 255


@pytest.mark.parametrize("sigmoid,groups,topk_groups,group_top", [(False, 1, 1, 1), (True, 4, 2, 2),
                                                                 (False, 4, 3, 1), (True, 2, 1, 2)])
def test_route_matches_brute_force(sigmoid, groups, topk_groups, group_top):
    rng = np.random.default_rng(4)
    lg = rng.normal(size=(6, 8)).astype(np.float32)
    bias = rng.normal(size=8) * 0.3
    ids, w = w8.route_scored(lg, 2, sigmoid, bias, groups, topk_groups, group_top)
    for t in range(6):
        x = torch.from_numpy(lg[t]).double()
        s = (torch.sigmoid(x) if sigmoid else torch.softmax(x, 0)).numpy()
        c, per = s + bias, 8 // groups
        worth = [np.sort(c[g * per:(g + 1) * per])[::-1][:group_top].sum() for g in range(groups)]
        best = max(itertools.combinations(range(groups), topk_groups), key=lambda q: sum(worth[g] for g in q))
        allowed = [e for e in range(8) if e // per in best]
        pair = max(itertools.permutations(allowed, 2), key=lambda q: (c[q[0]], c[q[1]]))
        assert tuple(ids[t]) == pair
        np.testing.assert_allclose(w[t], s[list(pair)] / s[list(pair)].sum(), rtol=1e-12)


def test_route_masked_rows_and_ties():
    lg = np.zeros((3, 6), dtype=np.float32)
    lg[0, :] = -np.inf
    lg[1, [0, 2, 3, 4, 5]] = [np.nan, -np.inf, -np.inf, -np.inf, np.nan]
    ids, w = w8.route_scored(lg, 3)
    assert list(ids[0]) == [0, 1, 2] and not w[0].any()
    assert list(ids[1]) == [1, 0, 2] and list(w[1]) == [1, 0, 0]
    assert list(ids[2]) == [0, 1, 2] and np.allclose(w[2], 1 / 3)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_matches_differences(sigmoid, renorm):
    rng = np.random.default_rng(5)
    lg = rng.normal(size=(3, 7))
    dw = rng.normal(size=(3, 3))
    ids, w = w8.route_scored(lg, 3, sigmoid, renorm=renorm, scale=1.5)
    got = w8.route_scored_grad(lg, ids, w, dw, sigmoid, renorm, 1.5)

    def loss(x):
        total = 0.0
        for t in range(3):
            s = w8.scores(x[t], sigmoid)[ids[t]]
            total += (dw[t] * 1.5 * (s / s.sum() if renorm else s)).sum()
        return total
    h = 1e-6
    for t, e in itertools.product(range(3), range(7)):
        d = np.zeros_like(lg)
        d[t, e] = h
        assert abs((loss(lg + d) - loss(lg - d)) / (2 * h) - got[t, e]) < 1e-8
