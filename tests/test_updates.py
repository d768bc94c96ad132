"""Orthogonalised updates against their definition in 64 bits, and their
refusals.

Bounds.  How far roundings are amplified depends on the matrix, and is measured
on it with a form in f32: stored values are f32, and a sum of products is taken
one term at a time, acc = f32(acc + a b).  The kernel's roundings, against that
form's: a stored value has 22 bits where f32 has 24, so each of these roundings is
at most 4 times as large; and a sum takes at most three additions (hi hi, hi lo, lo
hi) for each term, in whatever order the matrix instructions add their 16 terms,
each off by at most half a step of a partial sum: at most 3 times as much.  Where
the form is off by some error from 64 bits, the kernel may therefore be off by 4
times that, and by 2^-22 of the result for what it leaves out (lo lo, at most 2^-22
of a product); in the largest element by 4 times the form's and 2^-20 of the
result's largest (a largest error of few roundings is less even).
(A form whose sums are taken in another order says nothing about this: a CPU's
product of 2047 x 1990 by its transpose keeps many partial sums, and is off by
several times less than additions in a row.)
Results add half a step (bf16 2^-8, f32 2^-24)."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

import dnn_conv2d_bwd_amd as cbd

TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
USUAL = (3.4445, -4.7750, 2.0315)


def exact_product(a, b):
    return a @ b


def f32_product(a, b):
    """In f32, one term at a time."""
    acc = torch.zeros(a.shape[0], a.shape[1], b.shape[2], dtype=torch.float32, device=a.device)
    a, b = a.double(), b.double()
    for k in range(a.shape[2]):
        acc = torch.addcmul(acc.double(), a[:, :, k:k + 1], b[:, k:k + 1]).float()
    return acc


def define(m, steps=5, coefficients=None, eps=1e-7, scale=1.0, f32=False):
    norm = m.double().square().sum((1, 2), keepdim=True).sqrt() + eps
    x = m.double() / norm
    if f32:
        x = x.float()
    product = f32_product if f32 else exact_product
    flip = m.shape[1] > m.shape[2]
    x = x.transpose(1, 2).contiguous() if flip else x
    for k in range(steps):
        a, b, c = USUAL if coefficients is None else coefficients[k]
        q = product(x, x.transpose(1, 2).contiguous())
        p = b * q + c * product(q, q)
        x = a * x + product(p, x)
    return (scale * x).transpose(1, 2) if flip else scale * x


def draw(n, rows, cols, dtype="f32", seed=0, rank=None, scale=1e-3):
    gen = torch.Generator().manual_seed(4000 + seed)
    m = torch.randn(n, rows, cols, generator=gen)
    if rank:
        m = 0.3 * m + torch.randn(n, rows, rank, generator=gen) @ torch.randn(n, rank, cols, generator=gen) / rank ** 0.5
    return (scale * m).to(TORCH[dtype])


def near(got, m, dtype, name="", **kw):
    m = m.cuda()  # for the form's many small steps
    want, plain = define(m, **kw).cpu(), define(m, f32=True, **kw).double().cpu()
    got, half = got.double().cpu(), torch.finfo(TORCH[dtype]).eps / 2
    for i in range(m.shape[0]):
        w, err, err32 = want[i], (got[i] - want[i]).abs(), (plain[i] - want[i]).abs()
        ok = 4 * err32.norm() + (2.0 ** -22 + half) * w.norm()
        assert err.norm() <= ok, f"{name} matrix {i}: {float(err.norm() / w.norm())} off, {float(ok / w.norm())} allowed"
        top = w.abs().max()
        assert (err <= 4 * err32.max() + 2.0 ** -20 * top + half * w.abs()).all(), f"{name} matrix {i}: an element is off"


class Stack:
    """Matrices in a buffer with `gap` extra elements a row, `space` more rows
    between matrices and `off` elements before, NaN in all of them."""

    def __init__(self, m, gap=0, space=0, off=0):
        self.shape = n, r, c = m.shape
        pitch, mat = c + gap, (r + space) * (c + gap)
        self.buf = torch.full((off + n * mat + 64,), float("nan"), dtype=m.dtype, device="cuda")
        self.t = self.buf[off:off + n * mat].view(n, r + space, pitch)[:, :r, :c]
        self.t.copy_(m)

    def take(self):
        res = self.t.clone()
        self.t.fill_(float("nan"))
        assert bool(torch.isnan(self.buf).all()), "a store outside the output"
        return res


def call(m, gap=0, space=0, off=0, stream=None, **kw):
    p = cbd.ortho_plan(*m.shape, dtype="f32" if m.dtype == torch.float32 else "bf16", **kw)
    a, o = Stack(m, gap, space, off), Stack(torch.full(m.shape, float("nan"), dtype=m.dtype), gap, space, off)
    ws = torch.full((p.workspace_size() + 256,), 0xff, dtype=torch.uint8, device="cuda")  # NaN, and a guard
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    assert cbd.orthogonalize(p, a.t, o.t, ws[:p.workspace_size()], stream=stream) is o.t
    torch.cuda.synchronize()
    assert bool((ws[p.workspace_size():] == 0xff).all())
    return o.take()


# One element; vectors; sides around the runs of 32 and the tiles of 64 and 128; tall, wide, square; many.
SIZES = [(1, 1, 1), (3, 1, 40), (2, 40, 1), (5, 16, 16), (2, 31, 33), (3, 64, 64), (2, 65, 200), (2, 200, 65), (1, 128, 129),
         (70, 17, 24), (2, 96, 515), (1, 515, 389), (1, 300, 1030)]


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_against_definition(dtype, size):
    print("[ortho]", dtype, size, flush=True)
    m = draw(*size, dtype=dtype, seed=sum(size))
    near(call(m), m, dtype, str(size))


# matrices, rows, cols; tiles of A and B, and of X, where the last matrices have
# others both.  128 also with more tiles than
# compute units (two workgroups on one).
TILES = [((300, 64, 96), 64, 64), ((9, 512, 768), 64, 128), ((9, 700, 1100), 128, 128), ((17, 1500, 500), 128, 256),
         ((1, 2047, 1990), 128, 128), ((14, 1030, 1900), 128, 128), ((7, 1000, 2040), 128, 256),
         ((25, 1090, 1000), 256, 256), ((30, 1000, 1010), (256, 128), 256), ((32, 512, 1408), 64, (256, 128))]


@pytest.mark.gpu
@pytest.mark.parametrize("size,symmetric,step", TILES, ids=str)
def test_every_tile(size, symmetric, step):
    """Sizes at which each tile is chosen, with edges inside tiles."""
    info = cbd.ortho_plan(*size).info()
    print("[ortho] tiles", size, info.tile_symmetric, info.tile_step, flush=True)
    tiles = (info.tile_symmetric, info.tile_symmetric_rest), (info.tile_step, info.tile_step_rest)
    assert tiles == tuple(t if isinstance(t, tuple) else (t, 0) for t in (symmetric, step))
    m = draw(*size, seed=size[1], rank=max(1, min(size[1:]) // 8))
    got = call(m, steps=3)
    some = [0, size[0] - 1] if size[0] > 1 else [0]
    near(got[some], m[some], "f32", str(size), steps=3)


# A few tiles of A and a long contracted side, whose slices are joined: an edge
# inside the last slice, a last slice of one run, more than one matrix.
SLICED = [(1, 256, 4096), (1, 16, 4096), (1, 5, 8200), (3, 40, 2047), (1, 3000, 70), (2, 130, 3001), (5, 321, 2081), (1, 1, 65536)]


@pytest.mark.gpu
@pytest.mark.parametrize("size", SLICED, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slices(dtype, size):
    print("[ortho] slices", dtype, size, flush=True)
    assert cbd.ortho_plan(*size).info().slices > 1
    m = draw(*size, dtype=dtype, seed=size[1])
    near(call(m, steps=3), m, dtype, str(size), steps=3)


def near_in_parts(got, m, dtype, part, name="", steps=5, coarse=False):
    """near's bound for each half of the rows (or columns) by itself, and what a
    value that is small next to its matrix loses.

    A stored value is off by at most 2^-50 of the plan's bound (bf16 with tiles of
    256: 2^-39), where that is more than 2^-22 of itself; the bounds are at most 2 for X and A, 4 for B (powers of
    two above 1.21, 1.46 and 3.45).  In a row of the smaller side that adds to a
    step's result (norms, with |X| and |A| at most 1.46): sqrt(l) 2^-49 for X
    itself; sqrt(s) 2^-49 times |b + 2 c A| <= 10.8 for A, and sqrt(s) 2^-48 for B,
    both times |X|: sqrt(s) 2^-49 (10.8 + 2) 1.21.  A step makes at most 3.45
    times as much of it.  A column has the same bound with the sides exchanged, so
    both are taken."""
    m = m.cuda()
    want, plain = define(m, steps=steps).cpu(), define(m, steps=steps, f32=True).double().cpu()
    got, half = got.double().cpu(), torch.finfo(TORCH[dtype]).eps / 2
    s, l = min(m.shape[1:]), max(m.shape[1:])
    floor = sum(3.45 ** k for k in range(steps + 1)) * 2.0 ** -49 * (l ** 0.5 + 15.5 * (s ** 0.5 + l ** 0.5))
    floor *= 2.0 ** 11 if coarse else 1.0
    n = m.shape[part + 1] // 2
    for i in range(m.shape[0]):
        for at in (slice(0, n), slice(n, None)):
            w, g, p = ((v[i][at] if part == 0 else v[i][:, at]) for v in (want, got, plain))
            ok = 4 * (p - w).norm() + (2.0 ** -22 + half) * w.norm() + floor * w.shape[part] ** 0.5
            err = (g - w).norm()
            assert err <= ok, f"{name} matrix {i}, {at}: {float(err / w.norm())} off, {float(ok / w.norm())} allowed"


# Tiles of 64, of 64 in slices, of 128 with one and with two a unit, of 256, both ways.
PARTED = [(2, 256, 512), (2, 200, 64), (1, 100, 3000), (9, 700, 1100), (20, 700, 600), (25, 1090, 1000), (32, 512, 1408)]


@pytest.mark.gpu
@pytest.mark.parametrize("small,dtype", [(1e-4, "f32"), (1e-6, "f32"), (1e-5, "bf16"), (1e-8, "bf16")])
@pytest.mark.parametrize("size", PARTED, ids=str)
def test_rows_and_columns_of_different_size(size, small, dtype):
    """Rows that a gradient seldom reaches keep an accuracy of their own."""
    for part in (0, 1):
        print("[ortho] parts", size, small, part, dtype, flush=True)
        m = draw(*size, seed=size[1])
        (m[:, size[1] // 2:] if part == 0 else m[:, :, size[2] // 2:]).mul_(small)
        m = m.to(TORCH[dtype])
        some, steps, i = [0, size[0] - 1][:size[0]], 5 if min(size[1:]) < 500 else 3, cbd.ortho_plan(*size, dtype).info()
        tiles = i.tile_symmetric, i.tile_symmetric_rest, i.tile_step, i.tile_step_rest
        near_in_parts(call(m, steps=steps)[some], m[some], dtype, part, f"{size} {small} {part}", steps, dtype == "bf16" and 256 in tiles)


@pytest.mark.gpu
@pytest.mark.parametrize("gap,space,off", [(8, 0, 0), (1, 0, 1), (0, 3, 0), (5, 2, 3)])
def test_strides_and_alignment(gap, space, off):
    for dtype in ("bf16", "f32"):
        for size in ((3, 40, 72), (2, 101, 67)):
            m = draw(*size, dtype=dtype)
            got = call(m, gap, space, off)
            near(got, m, dtype)
            assert torch.equal(got, call(m))


@pytest.mark.gpu
@pytest.mark.parametrize("steps,coefficients", [
    (1, None), (3, None), (8, None), (2, [(1.5, -0.5, 0.0)]), (7, [(1.875, -1.25, 0.375)]),
    (3, [(8.2872, -23.5959, 17.3004), (4.1071, -2.9478, 0.5448), (3.9487, -2.9089, 0.5518)])])
def test_steps_and_coefficients(steps, coefficients):
    m = draw(2, 90, 140, rank=12)
    co = None if coefficients is None else coefficients * (steps if len(coefficients) == 1 else 1)
    near(call(m, steps=steps, coefficients=coefficients), m, "f32", steps=steps, coefficients=co)


@pytest.mark.gpu
def test_scale_and_eps():
    m = draw(2, 50, 70)
    near(call(m, scale=-0.2), m, "f32", scale=-0.2)
    near(call(m, eps=0.5), m, "f32", eps=0.5)
    for by in (1e-30, 1e-4, 1e30):  # the norm's squares are in 64 bits
        near(call(m * by, eps=1e-38), m * by, "f32", eps=1e-38)


@pytest.mark.gpu
def test_small_scales():
    """Down to results that are just normal numbers."""
    m = draw(2, 20, 30)
    for scale in (3e-30, 3e-36, -7e-36):
        near(call(m, scale=scale), m, "f32", scale=scale)


@pytest.mark.gpu
def test_known_results():
    """Matrices whose singular values are all alike come out as multiples of
    themselves: signed permutations, and a Hadamard matrix."""
    n = 64
    h = torch.ones(1, 1)
    while h.shape[0] < n:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)])
    perm = torch.eye(n)[torch.randperm(n, generator=torch.Generator().manual_seed(1))]
    m = torch.stack([h, 3.0 * perm, -0.01 * perm])
    x = 1.0 / (1.0 + 1e-7 / m.double().square().sum((1, 2)).sqrt()) / math.sqrt(n)
    for _ in range(5):
        x = USUAL[0] * x + USUAL[1] * x ** 3 + USUAL[2] * x ** 5
    want = torch.stack([h / 8, perm, -perm]).double() * x.view(3, 1, 1)
    # Each step's derivative is at most 3.95 in size, and each is off by at most
    # 16 roundings of 2^-22 of values up to 14.5: 14.5 * 16 * (1 + ... + 3.95^4) roundings.
    assert (call(m).double().cpu() - want).abs().max() <= 14.5 * 16 * 325 * 2.0 ** -22 * float(x.max()) / 8


@pytest.mark.gpu
def test_extremes():
    m = draw(5, 40, 56)
    m[1] = 0.0
    m[2, 3, 4] = float("nan")
    m[3, 0, 0] = float("inf")
    got = call(m)
    assert not got[1].any() and torch.isnan(got[2]).all() and torch.isnan(got[3]).all()
    keep = [0, 4]
    near(got[keep], m[keep], "f32")
    assert torch.equal(got[keep], call(m[keep]))
    one = torch.zeros(1, 33, 65)
    one[0, 32, 64] = 5.0  # a single element: its singular value is 1
    near(call(one), one, "f32")


@pytest.mark.gpu
def test_zeros_whatever_eps_is():
    m = draw(3, 20, 30)
    m[1] = 0.0
    for eps in (1e-300, 1e-310, 5e-324):
        got = call(m, eps=eps)
        assert torch.equal(got[1], torch.zeros_like(got[1])) and torch.isfinite(got).all()
        near(got[[0, 2]], m[[0, 2]], "f32", eps=eps)


@pytest.mark.gpu
def test_powers_of_two_cancel():
    """Also where the factor to the norm, or the norm's square, is past f32."""
    for dtype in ("f32", "bf16"):
        m = draw(3, 48, 70, dtype=dtype, scale=1.0)
        m[1] = 0.0
        want = call(m, eps=1e-300)
        assert not want[1].any() and bool(want[0].any())
        for power in (-110, -60, 100):  # (the smallest elements stay normal)
            m2 = torch.where(m.float().abs() < 2.0 ** -14, torch.zeros_like(m), m)
            assert torch.equal(call(m2.double().mul(2.0 ** power).to(m.dtype), eps=1e-300), call(m2, eps=1e-300)), power


@pytest.mark.gpu
def test_in_place_streams_repeats_and_graph_replays():
    m = draw(4, 100, 180, dtype="bf16")
    want = call(m)
    s = torch.cuda.Stream()
    for stream in (None, s, s):
        assert torch.equal(call(m, stream=stream), want)
    p = cbd.ortho_plan(4, 100, 180, "bf16")
    x = m.cuda()
    assert cbd.orthogonalize(p, x, out=x) is x and torch.equal(x, want)
    with pytest.raises(cbd.CbdError, match="overlaps"):
        wide = torch.zeros(4, 100, 190, dtype=torch.bfloat16, device="cuda")
        cbd.orthogonalize(p, wide[:, :, :180], out=wide[:, :, 10:])
    x = m.cuda()
    out, ws = torch.empty_like(x), torch.empty(p.workspace_size(), dtype=torch.uint8, device="cuda")
    cbd.orthogonalize(p, x, out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cbd.orthogonalize(p, x, out, ws)
    for i in range(4):
        x.copy_(draw(4, 100, 180, dtype="bf16", seed=i + 1))
        ws.fill_(0xff)
        graph.replay()
        torch.cuda.synchronize()
        mine = out.clone()
        torch.cuda.synchronize()
        assert torch.equal(mine, cbd.orthogonalize(p, x)), i


@pytest.mark.gpu
def test_convenience_and_written():
    m = draw(6, 40, 24).cuda()
    want = cbd.orthogonalize(cbd.ortho_plan(6, 40, 24), m)
    assert torch.equal(cbd.orthogonalized(m), want)
    assert torch.equal(cbd.orthogonalized(m.view(2, 3, 40, 24)), want.view(2, 3, 40, 24))
    assert torch.equal(cbd.orthogonalized(m[1]), want[1])
    assert torch.equal(cbd.orthogonalized(m[::2]), want[::2])
    assert cbd.orthogonalized(m[:0]).shape == (0, 40, 24)
    t = torch.zeros_like(m)
    loss = (torch.ones_like(t, requires_grad=True) * t).sum()
    cbd.orthogonalize(cbd.ortho_plan(6, 40, 24), m, out=t)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()


# ------------------------------------------------------------ refusals (CPU)

@pytest.mark.parametrize("over,status", [
    (dict(matrices=-1), 1), (dict(rows=0), 1), (dict(cols=-2), 1), (dict(dtype=2), 1), (dict(steps=0), 1),
    (dict(steps=65), 1), (dict(eps=0.0), 1), (dict(eps=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(matrices=65536), 2), (dict(rows=65537), 2), (dict(cols=65537), 2), (dict(matrices=65535, rows=65536, cols=65536), 2), (dict(matrices=0), 0), (dict(), 0),
    (dict(co=(3.0, float("nan"), 1.0)), 1), (dict(co=(0.0, 0.0, 0.0)), 2), (dict(co=(9.0, 9.0, 9.0)), 2),
    (dict(co=(1e-30, 0.0, 0.0)), 2), (dict(co=(1.5, -0.5, 0.0)), 0)])
def test_plan_refusals(over, status):
    kw = dict(matrices=2, rows=16, cols=24, dtype=cbd.F32, steps=5, eps=1e-7, scale=1.0)
    co = over.pop("co", None)
    kw.update(over)
    if co:
        kw["coefficients"] = (ctypes.c_double * 15)(*(co * 5))
    h = ctypes.c_void_p()
    assert cbd._lib.cbd_ortho_plan(ctypes.byref(cbd.OrthoProblem(**kw)), ctypes.byref(h)) == status
    assert bool(h.value) == (status == 0)
    if status:
        assert cbd._lib.cbd_last_error()
    cbd._lib.cbd_ortho_plan_destroy(h)


def test_run_refusals():
    """Argument checks come before any launch, so made-up addresses do."""
    S = cbd.OrthoStrides
    p = cbd.ortho_plan(3, 16, 24)
    i, o, ws, size = 0x10000, 0x20000, 0x1000000, p.workspace_size()

    def run(i=i, o=o, ws=ws, size=size, s=None, plan=p._h):
        return cbd._lib.cbd_orthogonalize(plan, i, o, ctypes.byref(s) if s else None, ws, size, None)

    assert run(plan=None) == 1 and run(i=None) == 1 and run(o=None) == 1 and run(ws=None) == 1
    assert run(size=size - 1) == 1 and run(ws=ws + 128) == 2
    assert run(i=i + 2) == 2 and run(o=o + 1) == 2
    assert run(s=S(23, 0, 0, 0)) == 1 and run(s=S(0, 0, 23, 0)) == 1 and run(s=S(0, 383, 0, 0)) == 1
    assert run(s=S(0, 0, 0, -1)) == 1 and run(s=S(2 ** 31 + 1, 0, 0, 0)) == 2 and run(s=S(0, 2 ** 40 + 1, 0, 0)) == 2
    assert run(o=i + 4) == 1 and run(o=i, s=S(24, 384, 32, 512)) == 1 and run(o=ws) == 1 and run(i=ws + 64) == 1
    none = cbd.ortho_plan(0, 16, 24)
    assert run(plan=none._h, i=None, o=None, ws=None, size=0) == 0


def test_info():
    i = cbd.ortho_plan(8, 4096, 2048, steps=5).info()
    assert (i.tile_symmetric, i.tile_symmetric_rest, i.tile_step, i.tile_step_rest) == (256, 128, 256, 0)
    assert i.launches == 2 + 5 * 5 and cbd.ortho_plan(8, 64, 64, steps=2).info().launches == 2 + 2 * 3
    assert i.flops == 8 * 5 * (3 * 2048 * 2048 * 4096 + 2048 ** 3)
    assert cbd.ortho_plan(0, 16, 16).info().launches == 0
    i = cbd.ortho_plan(1, 256, 4096, steps=5).info()
    assert (i.tile_symmetric, i.slices, i.launches) == (64, 16, 2 + 5 * 4) and cbd.ortho_plan(8, 64, 64).info().slices == 1


def test_range_of_the_usual_coefficients():
    """What ortho_plan's description says of five steps: singular values above 0.01
    of the norm end between 0.68 and 1.14."""
    x = torch.linspace(0.01, 1.0, 1000001, dtype=torch.float64)
    for _ in range(5):
        x = USUAL[0] * x + USUAL[1] * x ** 3 + USUAL[2] * x ** 5
    assert 0.68 <= float(x.min()) < 0.69 and 1.13 < float(x.max()) <= 1.14
    assert "0.68 and 1.14" in " ".join(cbd.ortho_plan.__doc__.split())


def test_python_refusals_without_a_gpu():
    with pytest.raises(ValueError, match="GPU"):
        cbd.orthogonalize(cbd.ortho_plan(1, 4, 4), torch.zeros(1, 4, 4))
    with pytest.raises(ValueError, match="triples"):
        cbd.ortho_plan(1, 4, 4, coefficients=[(1.0, 2.0)])
    with pytest.raises(ValueError, match="triples"):
        cbd.ortho_plan(1, 4, 4, coefficients=[(1.5, -0.5, 0.0)] * 4)
    with pytest.raises(ValueError, match="matrices"):
        cbd.orthogonalized(torch.zeros(4))
    with pytest.raises(ValueError, match="bfloat16"):
        cbd.orthogonalized(torch.zeros(4, 4, dtype=torch.float64))


def test_what_autograd_would_lose_is_refused():
    p = cbd.ortho_plan(1, 4, 4)
    m = torch.zeros(1, 4, 4, requires_grad=True)
    for call_ in (lambda: cbd.orthogonalize(p, m), lambda: cbd.orthogonalized(m), lambda: cbd.orthogonalized(m[0])):
        with pytest.raises(ValueError, match="autograd"):
            call_()
        with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
            call_()
    import torch.autograd.forward_ad as forward

    with forward.dual_level():
        dual = forward.make_dual(m.detach(), torch.ones(1, 4, 4))
        with pytest.raises(ValueError, match="tangent"):
            cbd.orthogonalize(p, dual)


def test_coefficients_that_are_no_triples_are_refused():
    """Also where there are three numbers a step all together."""
    for steps, co in ((2, [(1.0, 2.0)] * 3), (2, [(1.5, -0.5, 0.0, 1.5, -0.5, 0.0)]), (1, [(1.5,), (-0.5,), (0.0,)]),
                      (3, [(1.5, -0.5, 0.0)] * 2)):
        with pytest.raises(ValueError, match="triples"):
            cbd.ortho_plan(1, 4, 4, steps=steps, coefficients=co)
    assert cbd.ortho_plan(1, 4, 4, steps=2, coefficients=[(1.5, -0.5, 0.0)] * 2).steps == 2


@pytest.mark.gpu
def test_python_refusals():
    p = cbd.ortho_plan(2, 4, 8)
    m = torch.zeros(2, 4, 8, device="cuda")
    for bad in (m.bfloat16(), m[:1], m[:, :, :7], m.transpose(1, 2), m[:1].expand(2, 4, 8)):
        with pytest.raises(ValueError):
            cbd.orthogonalize(p, bad)
    with pytest.raises(ValueError):
        cbd.orthogonalize(p, m, out=torch.zeros(2, 4, 8))
    with pytest.raises(cbd.CbdError, match="workspace"):
        cbd.orthogonalize(p, m, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
