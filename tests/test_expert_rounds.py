"""Workgroups of the expert products that take several tiles, at both tile
sizes and through every way in and out of LDS, against the definition in 64
bits (bounds as in test_experts); and rows and experts that stay apart in every
kernel."""
from __future__ import annotations

import pytest
import torch

import dnn_conv2d_bwd_amd as cbd

from test_expert_kernels import on_gpu
from test_experts import ALL, TORCH, Call, close, split

MFMA = cbd.EXPERT_KERNEL_MFMA


def compare(call, n, tile, op, accumulate=None):
    assert call.plan.info({"forward": cbd.FORWARD, "bwd_data": cbd.BWD_DATA, "bwd_weight": cbd.BWD_WEIGHT}[op]).tile_m == tile
    want, mass = on_gpu(call)
    if accumulate is None:
        close(call(), want, mass, n, call.out_dtype, op)
    else:
        old = accumulate.double()
        close(call(accumulate=old), want + old, mass + old.abs() + want.abs(), n + 1, call.out_dtype, op)


# 128 x 128 tiles, more of them than the 512 workgroups that stay, of experts
# without rows, with few and with many, and rows of nobody's.  Widths: whole
# chunks; odd outputs (16-byte loads, any store); odd inputs and shifted starts
# (loads through registers); rows inside wider buffers.
@pytest.mark.gpu
@pytest.mark.parametrize("op,lay", [a for a in ALL if a[0] != "bwd_weight"])
@pytest.mark.parametrize("wide_in,wide_out,gap,off", [(200, 1000, 0, 0), (200, 1003, 0, 0), (203, 1001, 0, 0),
                                                      (328, 1000, 0, 1), (200, 1000, 8, 8), (203, 1003, 5, 0)])
def test_rounds_of_small_tiles(op, lay, wide_in, wide_out, gap, off):
    print("[expert]", op, lay, wide_in, wide_out, gap, off, flush=True)
    c, k = (wide_in, wide_out) if op == "forward" else (wide_out, wide_in)
    t = 12000
    ends = [0, 4000, 4001, 4001, 4100, 4400, 9000, 9000, 11000, 11700]
    compare(Call(op, lay, t, len(ends), c, k, ends, gap=gap, off=off, kernel=MFMA), wide_in, 128, op)


@pytest.mark.gpu
@pytest.mark.parametrize("lay", ["ekc", "eck"])
@pytest.mark.parametrize("dw", ["f32", "bf16"])
@pytest.mark.parametrize("c,k,off", [(1000, 520, 0), (1001, 519, 0), (1000, 520, 1)])
@pytest.mark.parametrize("add", [False, True])
def test_rounds_of_small_weight_gradients(lay, dw, c, k, off, add):
    print("[expert] bwd_weight", lay, dw, c, k, off, add, flush=True)
    t, e = 2500, 17
    ends = split(t - 7, e - 1, 4) + [t - 7]
    call = Call("bwd_weight", lay, t, e, c, k, ends, dw=dw, off=off, kernel=MFMA)
    old = torch.randn(*call.w.shape, generator=torch.Generator().manual_seed(2)).to(TORCH[dw]) if add else None
    compare(call, max(hi - lo for lo, hi in call.spans), 128, "bwd_weight", old)


# 256 x 256 tiles, six steps and more, a last feature tile that is partly used,
# up to and over the 64 experts whose rows stay in registers.
@pytest.mark.gpu
@pytest.mark.parametrize("op,lay", [a for a in ALL if a[0] != "bwd_weight"])
@pytest.mark.parametrize("t,e", [(17001, 3), (15003, 70)])
def test_rounds_of_large_tiles(op, lay, t, e):
    print("[expert]", op, lay, t, e, flush=True)
    wide_in, wide_out = 456, 2000
    c, k = (wide_in, wide_out) if op == "forward" else (wide_out, wide_in)
    compare(Call(op, lay, t, e, c, k, split(t - 5, e, 6), kernel=MFMA), wide_in, 256, op)


@pytest.mark.gpu
@pytest.mark.parametrize("e,c,k", [(36, 1000, 1024), (70, 520, 776)])
@pytest.mark.parametrize("dw,add", [("f32", False), ("f32", True), ("bf16", True)])
def test_rounds_of_large_weight_gradients(e, c, k, dw, add):
    print("[expert] bwd_weight", e, c, k, dw, add, flush=True)
    t = 250 * e
    call = Call("bwd_weight", "ekc", t, e, c, k, split(t - 9, e, 8), dw=dw, kernel=MFMA)
    old = torch.randn(*call.w.shape, generator=torch.Generator().manual_seed(2)).to(TORCH[dw]) if add else None
    compare(call, max(hi - lo for lo, hi in call.spans), 256, "bwd_weight", old)


KINDS = [("bf16", cbd.EXPERT_KERNEL_GENERIC), ("bf16", MFMA), ("bf16", cbd.EXPERT_KERNEL_STREAM),
         ("f32", cbd.EXPERT_KERNEL_AUTO)]


@pytest.mark.gpu
@pytest.mark.parametrize("c,k,off", [(72, 104, 0), (75, 101, 0), (72, 104, 1), (200, 136, 0), (197, 139, 3)])
@pytest.mark.parametrize("dtype,kernel", KINDS, ids=["generic", "mfma", "stream", "f32"])
@pytest.mark.parametrize("op,lay", ALL)
def test_rows_stay_apart_in_every_kernel(op, lay, dtype, kernel, c, k, off):
    """NaN and infinities in one expert's rows and weights reach no other
    expert's results (nor, for y and dx, any other row's)."""
    t, ends = 200, [45, 46, 130, 190]
    call = Call(op, lay, t, 4, c, k, ends, dtype=dtype, off=off, kernel=kernel)
    clean = call()
    for v in (call.x, call.dy):
        v[45] = float("nan")       # all of expert 1
        v[130:135] = float("inf")  # expert 3's first rows
        v[195] = float("nan")      # nobody's
    call.w[1] = float("nan")
    got = call()
    if op == "bwd_weight":
        assert torch.equal(got[[0, 2]], clean[[0, 2]])
        assert not torch.isfinite(got[1]).any() and not torch.isfinite(got[3]).any()
    else:
        keep = [i for i in range(t) if i != 45 and not 130 <= i < 135]
        assert torch.equal(got[keep], clean[keep])
        assert torch.isnan(got[45]).all() and (got[190:] == 0).all()
