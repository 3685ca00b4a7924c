"""The sizes of ``train_tiles`` reach the kernels that they are meant for, and all of them are
reached.  No GPU."""

import pytest

import int4_weight_only_amd as w4
import train_tiles as tt


def rows(T, k, E, N, K, B):
    return w4.w4_bf16_moe_gemm_tile(T, k, E, N, K, B), w4.w4_bf16_moe_gemm_workspace(T, k, E, N, K, B) > 0


def sums(T, k, E, N, K):
    return w4.w4_bf16_moe_wgrad_tile(T, k, E, N, K), w4.w4_bf16_moe_wgrad_workspace(T, k, E, N, K) > 0


def test_sizes_reach_their_kernels():
    for *sizes, tile, parts in tt.ROWS:
        assert rows(*sizes) == (tile, parts), sizes
    for *sizes, tile, parts in tt.SUMS:
        assert sums(*sizes) == (tile, parts), sizes
    for M, N, K, tile, parts in tt.DENSE:
        assert sums(M, 1, 1, N, K) == (tile, parts), (M, N, K)
        assert (w4.w4_bf16_gemm_tn_workspace(M, N, K) > 0) == parts
    for T, N, K, B, tile in tt.WIDE_ROWS:
        assert T * K >= 1 << 30 and rows(T, 1, 2, N, K, B)[0] == tile, (T, N, K)
    for T, N, K, transposed, tile in tt.WIDE_WEIGHTS:
        assert (N if transposed else min(N, 256)) * K >= 1 << 30 and rows(T, 1, 1, N, K, 64) == (tile, True)
    for T, E, N, K, codes, tile in tt.WIDE_SUMS:
        assert T * max(N, K) >= 1 << 30 and sums(T, 1, E, N, K)[0] == tile, (T, E, N, K)
    assert any(codes and T * K >= 1 << 31 for T, _, _, K, codes, _ in tt.WIDE_SUMS)


def test_every_kernel_is_reached():
    tiles = {(64, 64), (64, 128), (128, 128), (256, 256)}
    assert {c[-2] for c in tt.ROWS} == tiles
    assert {min(c[-2], (128, 256)) if c[-2][0] == 128 and c[-2][1] > 128 else c[-2] for c in tt.SUMS} == tiles | {(128, 256)}
    assert {c[-2] for c in tt.DENSE} == tiles | {(128, 256)}
    assert any(c[-1] for c in tt.ROWS) and any(c[-1] for c in tt.SUMS) and any(c[-1] for c in tt.DENSE)
    wide = {(64, 64): (64, 64), (64, 128): (64, 64), (128, 128): (128, 128), (256, 256): (256, 256)}
    assert {wide[c[-1]] for c in tt.WIDE_ROWS} == set(wide.values())
    # run bf16 and from codes where the codes are wide too
    for one in (True, False):
        assert {wide[c[-1]] for c in tt.WIDE_SUMS if (c[1] == 1) == one} == set(wide.values())


def test_tiles_of_invalid_sizes():
    for bad in ((-1, 1, 1, 8, 8, 64), (1, 1, 1, 8, 8, 32), (1, 1, 1025, 8, 8, 64), (1, 1, 1, 0, 8, 64)):
        with pytest.raises(ValueError):
            w4.w4_bf16_moe_gemm_tile(*bad)
    for bad in ((-1, 1, 1, 8, 8), (1, 0, 1, 8, 8), (1, 1, 1025, 8, 8), (1 << 29, 1, 1, 8, 8)):
        with pytest.raises(ValueError):
            w4.w4_bf16_moe_wgrad_tile(*bad)
    assert w4.w4_bf16_moe_gemm_tile(0, 1, 1, 8, 8, 64) == (0, 0)
