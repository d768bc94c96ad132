"""Every kernel of the expert layer, forced, at the sizes where its tiles and
steps begin and end, against the definition in 64 bits (bounds as in
test_experts)."""
from __future__ import annotations

import ctypes

import pytest
import torch

import dnn_conv2d_bwd_amd as cbd

from test_experts import ALL, TORCH, Call, close, split

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


def on_gpu(call, accumulate=None):
    """The definition in 64 bits on the GPU, where the CPU would take too long;
    (result, sum of |products|)."""
    x, dy, w = (v.double().cuda() for v in (call.x, call.dy, call.w))
    ekc = call.lay == "ekc"
    if call.op == "bwd_weight":
        want = torch.zeros_like(w)
        mass = torch.zeros_like(w)
        for i, (lo, hi) in enumerate(call.spans):
            a, b = (dy[lo:hi].t(), x[lo:hi]) if ekc else (x[lo:hi].t(), dy[lo:hi])
            want[i], mass[i] = a @ b, a.abs() @ b.abs()
    else:
        rows = x if call.op == "forward" else dy
        want = torch.zeros(call.t, call.k if call.op == "forward" else call.c, dtype=torch.float64, device="cuda")
        mass = torch.zeros_like(want)
        for i, (lo, hi) in enumerate(call.spans):
            m = w[i].t() if (call.op == "forward") == ekc else w[i]
            want[lo:hi], mass[lo:hi] = rows[lo:hi] @ m, rows[lo:hi].abs() @ m.abs()
    return want.cpu(), mass.cpu()


# Many tiles of 256 x 256: workgroups that take several, last rounds that are
# taken as halves, partial row tiles between whole ones.
@pytest.mark.gpu
@pytest.mark.parametrize("op,lay,c,k", [("forward", "ekc", 72, 2048), ("forward", "eck", 72, 2048),
                                        ("bwd_data", "ekc", 2048, 136), ("bwd_data", "eck", 2048, 136)])
@pytest.mark.parametrize("t,ends", [(16800, [16385, 16385, 16700]), (17000, [300, 8000, 17000]),
                                    (20000, [5000, 5100, 20000]), (16500, [16500, 16500, 16500])])
def test_rounds_of_large_tiles(op, lay, c, k, t, ends):
    print("[expert]", op, lay, t, ends, flush=True)
    call = Call(op, lay, t, 3, c, k, ends, kernel=cbd.EXPERT_KERNEL_MFMA)
    assert call.plan.info(cbd.FORWARD if op == "forward" else cbd.BWD_DATA).tile_m == 256
    want, mass = on_gpu(call)
    close(call(), want, mass, c if op == "forward" else k, "bf16", op)


@pytest.mark.gpu
@pytest.mark.parametrize("lay", ["ekc", "eck"])
@pytest.mark.parametrize("dw", ["f32", "bf16"])
@pytest.mark.parametrize("add", [False, True])
def test_large_weight_gradients(lay, dw, add):
    t, e, c, k = 500, 36, 1000, 1024
    ends = split(t, e, 5)
    call = Call("bwd_weight", lay, t, e, c, k, ends, dw=dw, kernel=cbd.EXPERT_KERNEL_MFMA)
    assert call.plan.info(cbd.BWD_WEIGHT).tile_m == 256
    print("[expert] bwd_weight", lay, dw, add, flush=True)
    want, mass = on_gpu(call)
    n = max(hi - lo for lo, hi in call.spans)
    if not add:
        return close(call(), want, mass, n, dw, "bwd_weight")
    old = torch.randn(*call.w.shape, generator=torch.Generator().manual_seed(2)).to(TORCH[dw]).double()
    close(call(accumulate=old), want + old, mass + old.abs() + want.abs(), n + 1, dw, "accumulate")
