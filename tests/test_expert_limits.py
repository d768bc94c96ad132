"""Launch limits of the expert layer: a grid has fewer than 2^32 threads, 256 a
workgroup.  A plan takes the kernel or the tile that stays below, and a call
whose tiles are too many is refused before it is launched."""
from __future__ import annotations

import pytest

import dnn_conv2d_bwd_amd as cbd

MOST = (2 ** 32 - 1) // 256


@pytest.mark.parametrize("kw", [
    # few rows an expert and many of them: weights that would stream
    dict(tokens=2 ** 20, experts=65536, c=16, k=8192, w_layout="ekc", dtype="bf16"),
    dict(tokens=2 ** 20, experts=65536, c=16, k=8192, w_layout="ekc", dtype="bf16",
         force_kernel=cbd.EXPERT_KERNEL_STREAM),
    # rows for more than 2^24 tiles of 64
    dict(tokens=2 ** 30, experts=1, c=1, k=1, dtype="f32"),
    dict(tokens=2 ** 30, experts=1, c=1, k=1, dtype="bf16", force_kernel=cbd.EXPERT_KERNEL_GENERIC),
    dict(tokens=2 ** 30, experts=4, c=4096, k=4096, dtype="bf16"),
])
def test_plans_stay_below(kw):
    p = cbd.expert_plan(**kw)
    for op in (cbd.FORWARD, cbd.BWD_DATA, cbd.BWD_WEIGHT):
        assert 0 < p.info(op).grid <= MOST


def test_small_tiles_up_to_the_limit():
    """The last size whose tiles of 64 fit, and the first whose do not."""
    rows = 64 * (MOST - 2)
    assert cbd.expert_plan(rows, 1, 1, 1, dtype="f32").info().tile_m == 64
    assert cbd.expert_plan(rows + 64, 1, 1, 1, dtype="f32").info().tile_m == 128


def test_too_many_tiles_are_refused():
    """Checks come before any launch, so made-up addresses do."""
    p = cbd.expert_plan(2 ** 30, 1, 1, 4096, dtype="f32")
    x, w, ends, y = 1 << 34, 1 << 41, 1 << 40, 1 << 46
    assert cbd._lib.cbd_expert_forward(p._h[32], x, w, ends, y, None, None) == 2
    assert b"too many tiles" in cbd._lib.cbd_last_error()
