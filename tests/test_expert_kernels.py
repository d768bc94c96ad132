"""Every kernel of the expert layer, forced, at the sizes where its tiles and
steps begin and end, against the definition in 64 bits (bounds as in
test_experts)."""
from __future__ import annotations

import ctypes

import pytest

import dnn_conv2d_bwd_amd as cbd

from test_experts import ALL, Call, split

KERNELS = [cbd.EXPERT_KERNEL_GENERIC, cbd.EXPERT_KERNEL_MFMA, cbd.EXPERT_KERNEL_STREAM]
NAMES = [cbd.EXPERT_KERNEL_NAMES[k] for k in KERNELS]

# rows, experts, c, k: contracted lengths around one step and the ring of
# stages, feature edges around the tiles, odd widths.
SIZES = [(5, 2, 8, 8), (70, 3, 32, 264), (129, 2, 40, 256), (257, 2, 96, 520), (300, 1, 104, 136), (513, 3, 256, 128),
         (640, 70, 136, 248), (90, 4, 33, 300), (200, 3, 259, 31), (1100, 5, 300, 77)]


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("op,lay", ALL)
@pytest.mark.parametrize("kernel", KERNELS, ids=NAMES)
def test_forced(kernel, op, lay, size):
    t, e, c, k = size
    print("[expert]", cbd.EXPERT_KERNEL_NAMES[kernel], op, lay, size, flush=True)
    for dw in ("f32", "bf16")[:2 if op == "bwd_weight" else 1]:
        Call(op, lay, t, e, c, k, split(t, e, seed=t), dw=dw, seed=t, kernel=kernel).check()


@pytest.mark.gpu
@pytest.mark.parametrize("gap,off", [(8, 0), (1, 3), (64, 8)])
@pytest.mark.parametrize("op,lay", ALL)
@pytest.mark.parametrize("kernel", KERNELS, ids=NAMES)
def test_forced_strides(kernel, op, lay, gap, off):
    print("[expert]", cbd.EXPERT_KERNEL_NAMES[kernel], op, lay, gap, off, flush=True)
    Call(op, lay, 330, 4, 296, 280, [10, 150, 151, 300], gap=gap, off=off, kernel=kernel).check()


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 31, 32, 33, 63, 65, 97, 127, 129, 161, 191, 193, 255, 256, 257])
@pytest.mark.parametrize("op,lay", ALL)
def test_row_blocks(op, lay, rows):
    """Expert sizes around the row blocks of a tile."""
    print("[expert]", op, lay, rows, flush=True)
    for kernel in KERNELS:
        Call(op, lay, 2 * rows + 3, 3, 64, 72, [rows, rows, 2 * rows], kernel=kernel).check()


def test_forced_kernels_refuse_f32():
    for kernel in KERNELS[1:]:
        prob = cbd.ExpertProblem(8, 2, 16, 16, cbd.EKC, cbd.F32, cbd.F32, 32)
        h = ctypes.c_void_p()
        assert cbd._lib.cbd_expert_plan(ctypes.byref(prob), ctypes.byref(cbd.ExpertOptions(kernel)),
                                        ctypes.byref(h)) == 2
        assert not h.value
