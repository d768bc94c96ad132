"""The norms around a block against their definition in 64 bits, and their
refusals.

Bounds, with e = 2^-24 (half a step of f32).  A sum over a row goes through at
most 64 additions on the way of any term (16 elements a thread, 6 steps of a
wave, 16 waves), so it is off by at most 64 e of the sum of magnitudes, and 1 /
rms by at most 40 e of itself (half of that, a division, a root).  The rest are
single operations, at most 8 of them between two sums.  With t = scale * gate *
w_post * yn, every bound below follows the formula term by term.  Results add
half a step of their type."""
from __future__ import annotations

import ctypes

import pytest
import torch

import dnn_conv2d_bwd_amd as cbd

TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
E = 2.0 ** -24
PARTS = ("r", "y", "w_post", "gate", "w_pre")


# ------------------------------------------------------------ definition

def inverse(v, eps):
    return 1.0 / (v.square().mean(1, keepdim=True) + eps).sqrt()


def define(a, eps, scale):
    """z, n, and the two factors, of a dict of 64-bit operands (None: left out)."""
    t = torch.zeros_like(a["r"])
    ry = rz = torch.ones_like(a["r"][:, :1])
    if a["y"] is not None:
        t = a["y"]
        if a["w_post"] is not None:
            ry = inverse(t, eps)
            t = t * ry * a["w_post"]
        t = scale * t if a["gate"] is None else scale * t * a["gate"]
    z = a["r"] + t
    n = None
    if a["w_pre"] is not None:
        rz = inverse(z, eps)
        n = z * rz * a["w_pre"]
    return z, n, ry, rz, t


def within(got, want, slack, dtype, name):
    tol = slack + torch.finfo(TORCH[dtype]).eps / 2 * (want.abs() + slack) + 1e-37
    err = (got.double().cpu() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol)[bad].max())} x"


class Block:
    """Operands on the host in 64 bits (values of the type), calls on device
    views with `gap` extra elements a row and `off` before them, NaN in both."""

    def __init__(self, rows, c, dtype="bf16", dw="f32", post=True, gate="channel", pre=True, y=True, eps=1e-6, scale=0.5,
                 gap=0, off=0, seed=0):
        gen = torch.Generator().manual_seed(3000 + seed)

        def draw(*shape, scale=1.0, mean=0.0):
            return (mean + scale * torch.randn(*shape, generator=gen)).to(TORCH[dtype]).double()

        self.rows, self.c, self.dtype, self.dw, self.gap, self.off = rows, c, dtype, dw, gap, off
        self.a = dict(r=draw(rows, c, scale=2.0), y=draw(rows, c, scale=0.7), w_post=draw(c, mean=1.0, scale=0.2),
                      gate=draw(c, mean=0.5, scale=0.5) if gate == "channel" else draw(rows, c),
                      w_pre=draw(c, mean=1.0, scale=0.3))
        for part, there in (("y", y), ("w_post", post and y), ("gate", gate != "none" and y), ("w_pre", pre)):
            if not there:
                self.a[part] = None
        self.dz, self.dn = draw(rows, c, scale=0.1), draw(rows, c, scale=0.1) if pre else None
        self.plan = cbd.block_plan(rows, c, dtype, dw, eps, scale)

    def view(self, fill=None):
        n = self.off + self.rows * (self.c + self.gap)
        buf = torch.full((n + 64,), float("nan"), dtype=TORCH[self.dtype], device="cuda")
        v = buf[self.off:n].view(self.rows, self.c + self.gap)[:, :self.c]
        if fill is not None:
            v.copy_(fill.to(TORCH[self.dtype]))
        return v, buf

    def device(self):
        return {k: None if v is None else v.to(TORCH[self.dtype]).cuda() if v.dim() == 1 else self.view(v)[0]
                for k, v in self.a.items()}

    def read(self, out, buf):
        torch.cuda.synchronize()
        res = out.clone()
        out.fill_(float("nan"))
        assert bool(torch.isnan(buf).all()), "a store outside the output"
        return res

    def forward(self, stream=None):
        d = self.device()
        z, zb = self.view() if d["y"] is not None else (None, None)
        n, nb = self.view() if d["w_pre"] is not None else (None, None)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        got = cbd.block_forward(self.plan, d["r"], d["y"], d["w_post"], d["gate"], d["w_pre"], save=True, z=z, n=n,
                                stream=stream)
        torch.cuda.synchronize()
        assert got[0] is z and got[1] is n
        return None if z is None else self.read(z, zb), None if n is None else self.read(n, nb), got[2].clone()

    def bwd(self, stream=None, mask=(True,) * 5, dz=True, dn=True):
        d = self.device()
        _, _, ry, rz, _ = define(self.a, self.plan.eps, self.plan.scale)
        stats = torch.cat([ry, rz], 1).float().cuda()
        outs = dict(dr=self.view())
        if d["y"] is not None:
            outs["dy"] = self.view()
        if d["gate"] is not None and d["gate"].dim() == 2:
            outs["dgate"] = self.view()
        dz = self.view(self.dz)[0] if dz else None
        dn = self.view(self.dn)[0] if dn and self.dn is not None else None
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        got = cbd.block_bwd(self.plan, dz, dn, d["r"], d["y"], stats, d["w_post"], d["gate"], d["w_pre"],
                            output_mask=mask, stream=stream, **{k: v[0] for k, v in outs.items()})
        torch.cuda.synchronize()
        got = [None if g is None else g for g in got]
        for i, k in ((0, "dr"), (1, "dy"), (3, "dgate")):
            if k in outs and got[i] is not None:
                assert got[i] is outs[k][0]
                got[i] = self.read(*outs[k])
        return got

    def check(self, bwd=True):
        a, eps, scale = self.a, self.plan.eps, self.plan.scale
        z, n, ry, rz, t = define(a, eps, scale)
        gz, gn, stats = self.forward()
        dt = 48 * E * t.abs()                      # t has one sum and a few operations
        dz_ = dt + E * z.abs() + E * a["r"].abs()
        if gz is not None:
            within(gz, z, dz_, self.dtype, "z")
        # 1 / rms of z moves with z by at most |dz| / |z| of itself.
        move = dz_.norm(dim=1, keepdim=True) / z.norm(dim=1, keepdim=True).clamp(min=1e-300)
        if n is not None:
            within(gn, n, (48 * E + move) * n.abs() + dz_ * (rz * a["w_pre"]).abs(), self.dtype, "n")
        within(stats[:, :1], ry, 40 * E * ry, "f32", "1 / rms of y")
        within(stats[:, 1:], rz, (40 * E + move) * rz, "f32", "1 / rms of z")
        if bwd:
            self.check_bwd()

    def check_bwd(self, use_dz=True, use_dn=True):
        a, eps, scale, C = self.a, self.plan.eps, self.plan.scale, self.c
        z, n, ry, rz, t = define(a, eps, scale)
        dz = self.dz if use_dz else torch.zeros_like(self.dz)
        dn = self.dn if use_dn and self.dn is not None else torch.zeros_like(self.dz)
        leaf = {k: None if v is None else v.clone().requires_grad_() for k, v in a.items()}
        outs = define(leaf, eps, scale)
        outs, grads = (outs[:2], (dz, dn)) if n is not None else (outs[:1], (dz,))
        want = [k for k in PARTS if leaf[k] is not None]
        ref = dict(zip(want, torch.autograd.grad(outs, [leaf[k] for k in want], grads, allow_unused=True)))
        got = dict(zip(PARTS, self.bwd(dz=use_dz, dn=use_dn)))
        assert all((got[k] is None) == (a[k] is None) for k in PARTS)

        def sums(v):
            return v.sum(1, keepdim=True) / C

        one = torch.ones(())
        w_post, w_pre = (one if a[k] is None else a[k].abs() for k in ("w_post", "w_pre"))
        gate = one if a["gate"] is None else a["gate"].abs()
        c = (abs(scale) * gate * w_post).expand_as(z)
        yn = (a["y"] * ry).abs() if a["y"] is not None else torch.zeros_like(z)
        zn, v = (z * rz).abs(), (dn * w_pre).abs() if n is not None else torch.zeros_like(z)
        d_zn = 8 * E * (a["r"].abs() + t.abs()) * rz
        along = rz * sums(v * zn)
        d_along = rz * sums(v * (64 * E * zn + d_zn)) + 4 * E * along
        e = dz.abs() + rz * v
        d_r = 8 * E * (e + along * zn) + zn * d_along + along * d_zn
        within(got["r"], ref["r"], d_r, self.dtype, "dr")
        dr = ref["r"].abs() + d_r
        if a["y"] is not None:
            back = sums(c * yn * e) + along * sums(c * yn * zn)
            d_back = 80 * E * back + d_along * sums(c * yn * zn) + along * sums(c * yn * d_zn)
            d_y = c * d_r + 8 * E * c * dr
            if a["w_post"] is not None:
                d_y = ry * (d_y + yn * d_back + 8 * E * yn * back)
            within(got["y"], ref["y"], d_y, self.dtype, "dy")
        deep = 64 + self.rows  # additions of a column's sum
        if a["w_pre"] is not None:
            within(got["w_pre"], ref["w_pre"], (dn.abs() * (d_zn + deep * E * zn)).sum(0), self.dw, "dw_pre")
        term = abs(scale) * yn * (d_r + 8 * E * dr)
        if a["w_post"] is not None:
            within(got["w_post"], ref["w_post"], (gate * (term + deep * E * abs(scale) * yn * dr)).sum(0), self.dw, "dw_post")
        if a["gate"] is not None and a["gate"].dim() == 1:
            within(got["gate"], ref["gate"], (w_post * (term + deep * E * abs(scale) * yn * dr)).sum(0), self.dw, "dgate")
        elif a["gate"] is not None:
            within(got["gate"], ref["gate"], w_post * term, self.dtype, "dgate")


FORMS = [dict(post=p, gate=g) for p in (True, False) for g in ("none", "channel", "row")]
# One element, one row, a wave's row, chunks that end inside, several waves, every number of lanes.
SIZES = [(1, 1), (3, 7), (5, 64), (1, 4096), (37, 515), (130, 512), (9, 1000), (70, 1025), (21, 2048), (6, 5001),
         (7, 8192), (3, 8200), (2, 16384), (2500, 40)]


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_against_definition(dtype, size):
    print("[block]", dtype, size, flush=True)
    form = FORMS[sum(size) % len(FORMS)]
    Block(*size, dtype=dtype, dw=dtype, seed=size[0]).check()
    Block(*size, dtype=dtype, seed=size[1], **form).check()


@pytest.mark.gpu
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("form", FORMS, ids=str)
def test_parts(form, pre):
    for dtype in ("bf16", "f32"):
        b = Block(33, 200, dtype=dtype, pre=pre, **form)
        b.check()
        b.check_bwd(use_dz=False)
        if pre:
            b.check_bwd(use_dn=False)


@pytest.mark.gpu
def test_norm_alone():
    for dtype in ("bf16", "f32"):
        b = Block(40, 136, dtype=dtype, y=False)
        b.check()
        b.check_bwd(use_dz=False)


@pytest.mark.gpu
@pytest.mark.parametrize("gap,off", [(8, 0), (1, 0), (0, 1), (3, 5), (64, 8)])
def test_strides_and_alignment(gap, off):
    for dtype in ("bf16", "f32"):
        for c in (72, 131, 1048):
            print("[block]", dtype, c, gap, off, flush=True)
            Block(29, c, dtype=dtype, gate="row", gap=gap, off=off).check()


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 0.5])
def test_scale_and_eps(eps, scale):
    Block(20, 300, dtype="f32", eps=eps, scale=scale).check()


@pytest.mark.gpu
def test_extreme_rows():
    """Zeros, tiny and huge values follow the formula; NaN and infinities stay
    in their row, but for the vectors' gradients that sum over rows."""
    for dtype in ("bf16", "f32"):
        b = Block(12, 96, dtype=dtype)
        b.a["r"][0], b.a["y"][0] = 0.0, 0.0
        b.a["r"][1], b.a["y"][1] = b.a["r"][1] * 2.0 ** -40, b.a["y"][1] * 2.0 ** -40
        b.a["r"][2], b.a["y"][2] = b.a["r"][2] * 2.0 ** 40, b.a["y"][2] * 2.0 ** 50
        b.check()
        clean, (dr, dy, *_) = b.forward(), b.bwd()
        b.a["y"][4], b.a["r"][7], b.dz[9] = float("nan"), float("inf"), float("nan")
        z, n, stats = b.forward()
        dr2, dy2, *_ = b.bwd()
        same = [i for i in range(12) if i not in (4, 7, 9)]
        for u, v in zip((*clean, dr, dy), (z, n, stats, dr2, dy2)):
            assert torch.equal(u[same], v[same])
        assert torch.equal(clean[0][9], z[9]) and not torch.isfinite(n[4]).any() and not torch.isfinite(dr2[9]).any()
    b = Block(3, 40, eps=0.0)
    b.a["y"][1] = 0.0  # 0 / 0, by the formula
    z, _, _ = b.forward()
    assert torch.isnan(z[1]).all() and torch.isfinite(z[[0, 2]]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,rows,c", [("bf16", 6, 96), ("f32", 700, 515), ("bf16", 700, 4096), ("bf16", 6, 8200), ("f32", 6, 8196)])
@pytest.mark.parametrize("form", FORMS, ids=str)
def test_a_norm_without_a_gradient_takes_no_part(form, dtype, rows, c):
    """Where n is not there, or has no gradient, r and w_pre are no part of the
    results: what they hold changes no bit, infinities and NaN included."""
    inf, nan = float("inf"), float("nan")
    print("[block]", form, dtype, rows, c, flush=True)
    without = Block(rows, c, dtype=dtype, pre=False, **form)
    want = without.bwd()
    assert torch.equal(want[0].double().cpu(), without.dz)
    without.a["r"][1], without.a["r"][2, 3], without.a["r"][4] = inf, nan, -inf
    b = Block(rows, c, dtype=dtype, **form)
    b.a["r"][1], b.a["r"][2, 3], b.a["r"][4], b.a["w_pre"][5] = inf, nan, -inf, inf
    for got in (without.bwd(), b.bwd(dn=False)):
        for u, v in zip(want[:4], got):
            assert (u is None) == (v is None) and (u is None or torch.equal(u, v))
    assert torch.equal(got[4], torch.zeros_like(got[4]))
    if not form["post"] and form["gate"] == "none":
        # dy is scale * dz: y is no part of it either.
        b.a["y"][3] = inf
        got = b.bwd(dn=False)
        assert all(torch.equal(u, v) for u, v in zip(want[:2], got)) and not got[4].any()


@pytest.mark.gpu
def test_a_norm_alone_without_a_gradient():
    for dtype, c in (("bf16", 72), ("f32", 8196)):
        b = Block(5, c, dtype=dtype, y=False)
        b.a["r"][1], b.a["w_pre"][0] = float("inf"), float("nan")
        dr, dy, _, _, dw = b.bwd(dn=False)
        assert torch.equal(dr.double().cpu(), b.dz) and dy is None and torch.equal(dw, torch.zeros_like(dw))


@pytest.mark.gpu
def test_in_place_is_the_same():
    b = Block(50, 600)
    d = b.device()
    p = b.plan
    args = (d["w_post"], d["gate"], d["w_pre"])
    z, n, stats = cbd.block_forward(p, d["r"], d["y"], *args, save=True)
    dz, dn = b.dz.bfloat16().cuda(), b.dn.bfloat16().cuda()
    want = cbd.block_bwd(p, dz, dn, d["r"], d["y"], stats, *args)
    got = cbd.block_bwd(p, dz, dn, d["r"], d["y"], stats, *args, dr=dz, dy=dn)
    assert got[0] is dz and got[1] is dn and all(torch.equal(u, v) for u, v in zip(got, want))
    z2, n2 = cbd.block_forward(p, d["r"], d["y"], *args, z=d["r"], n=d["y"])
    assert z2 is d["r"] and torch.equal(z, z2) and torch.equal(n, n2)
    wide = torch.zeros(50, 1200, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(z=wide[:, 1:601], n=wide[:, 600:]), dict(z=d["y"]), dict(n=d["r"]), dict(n=d["w_pre"].expand(50, 600))):
        with pytest.raises((cbd.CbdError, ValueError)):
            cbd.block_forward(p, d["r"], d["y"], *args, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,c", [("bf16", 8200), ("bf16", 12301), ("f32", 8190), ("f32", 8196), ("f32", 13001)])
def test_wide_rows(dtype, c):
    """More rows than workgroups, of widths that a thread reads twice; in place too."""
    for gate in ("row", "channel"):
        print("[block]", dtype, c, gate, flush=True)
        b = Block(300, c, dtype=dtype, gate=gate)
        b.check()
        d = b.device()
        args = (d["w_post"], d["gate"], d["w_pre"])
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        z, n, stats = cbd.block_forward(b.plan, d["r"], d["y"], *args, save=True)
        dz, dn = b.dz.to(dt).cuda(), b.dn.to(dt).cuda()
        want = cbd.block_bwd(b.plan, dz, dn, d["r"], d["y"], stats, *args)
        got = cbd.block_bwd(b.plan, dz, dn, d["r"], d["y"], stats, *args, dr=dz, dy=dn)
        assert got[0] is dz and got[1] is dn and all(torch.equal(u, v) for u, v in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,rows,c", [("bf16", 1 << 19, 4096), ("bf16", 1 << 22, 512), ("f32", 1 << 21, 512), ("bf16", 1 << 19, 8200),
                                          ("bf16", 1 << 24, 64)])
def test_sums_of_many_rows(dtype, rows, c):
    """A column's sum of equal terms just below 1, which one f32 sum of 2048 rows
    would take as 1 from the 512th on: 3 / 4 of 2.99e-5 off.  128 rows at a time,
    a term is in at most 128 additions of its thread's, one for each 128 rows, 32
    of a workgroup's and one rounding, each off by at most 2^-24 of the sum."""
    print("[block] many rows", dtype, rows, c, flush=True)
    p = cbd.block_plan(rows, c, dtype, "f32", scale=1 - 2.99e-5)
    ones = torch.ones(rows, c, dtype=TORCH[dtype], device="cuda")
    w, stats = torch.ones(c, dtype=TORCH[dtype], device="cuda"), torch.ones(rows, 2, device="cuda")
    stats[:, 1] = 1 - 2.99e-5
    tol = (128 + rows / 256 / 128 + 32 + 1) * 2.0 ** -24 * rows
    # zn = r / rms and dn = 1; then scale * dz * y.
    dw = cbd.block_bwd(p, None, ones, ones, stats=stats, w_pre=w, output_mask=(0, 0, 0, 0, 1))[4]
    assert float((dw.double() - rows * stats[0, 1].double()).abs().max()) <= tol
    dgate = cbd.block_bwd(p, ones, None, ones, ones, gate=w, output_mask=(0, 0, 0, 1, 0))[3]
    assert float((dgate.double() - rows * torch.tensor(p.scale).float().double().cuda()).abs().max()) <= tol


@pytest.mark.gpu
def test_masks_and_empty():
    b = Block(17, 80, gate="row")
    whole = b.bwd()
    for mask in ((1, 0, 0, 0, 0), (0, 1, 0, 0, 0), (0, 0, 1, 0, 0), (0, 0, 0, 1, 0), (0, 0, 0, 0, 1), (0, 0, 0, 0, 0)):
        part = b.bwd(mask=mask)
        assert all((v is None) == (not m) for v, m in zip(part, mask))
        assert all(torch.equal(u, v) for u, v, m in zip(whole, part, mask) if m)
    none = Block(0, 80)
    z, n, stats = none.forward()
    assert z.shape == n.shape == (0, 80) and stats.shape == (0, 2)
    dr, dy, *vectors = none.bwd()
    assert dr.shape == dy.shape == (0, 80) and all(v.shape == (80,) and not v.any() for v in vectors)


@pytest.mark.gpu
def test_no_rows_and_vectors_that_are_not_finite():
    none = Block(0, 80)
    none.a["gate"][3], none.a["w_post"][5], none.a["w_pre"][7] = float("inf"), float("nan"), float("inf")
    assert all(torch.equal(v, torch.zeros_like(v)) for v in none.bwd()[2:])


@pytest.mark.gpu
def test_streams_repeats_and_graph_replays():
    b = Block(700, 264)
    want = [*b.forward(), *b.bwd()]
    s = torch.cuda.Stream()
    for stream in (None, s, s):
        assert all(torch.equal(u, v) for u, v in zip([*b.forward(stream), *b.bwd(stream)], want))
    d, dz, dn = b.device(), b.dz.bfloat16().cuda(), b.dn.bfloat16().cuda()
    args = (d["w_post"], d["gate"], d["w_pre"])

    def call():
        z, n, stats = cbd.block_forward(b.plan, d["r"], d["y"], *args, save=True)
        return z, n, stats, *cbd.block_bwd(b.plan, dz, dn, d["r"], d["y"], stats, *args)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for i in range(4):
        d["r"].mul_(0.75)
        graph.replay()
        torch.cuda.synchronize()
        mine = [t.clone() for t in out]
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(mine, call())), i


# ------------------------------------------------------------ autograd

@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS, ids=str)
def test_autograd(form):
    """The recorded call's gradients are block_bwd's, all together and each
    alone; and, along a direction, what differences of the definition give."""
    b = Block(30, 2 * 48, dtype="f32", **form)
    d = {k: None if v is None else v.float().cuda() for k, v in b.a.items()}
    dz, dn = b.dz.float().cuda(), b.dn.float().cuda()
    there = [k for k in PARTS if d[k] is not None]
    z, n, stats = cbd.block_forward(b.plan, *(d[k] for k in PARTS), save=True)
    want = dict(zip(PARTS, cbd.block_bwd(b.plan, dz, dn, d["r"], d["y"], stats, d["w_post"], d["gate"], d["w_pre"])))
    for need in [there] + [[k] for k in there]:
        leaf = {k: None if v is None else v.clone().requires_grad_(k in need) for k, v in d.items()}
        zn = cbd.block_norm(leaf["r"].view(5, 6, 96), None if leaf["y"] is None else leaf["y"].view(5, 6, 96), leaf["w_post"],
                            leaf["gate"] if leaf["gate"] is None or leaf["gate"].dim() == 1 else leaf["gate"].view(5, 6, 96),
                            leaf["w_pre"], scale=0.5)
        assert torch.equal(zn[0].reshape(30, 96), z) and torch.equal(zn[1].reshape(30, 96), n)
        got = torch.autograd.grad(zn, [leaf[k] for k in need], (dz.view(5, 6, 96), dn.view(5, 6, 96)))
        assert all(torch.equal(g, want[k]) for g, k in zip(got, need)), need
    gen = torch.Generator().manual_seed(2)
    way = {k: None if v is None else torch.randn(v.shape, generator=gen, dtype=torch.float64) for k, v in b.a.items()}
    up, down = (define({k: None if v is None else v + s * 1e-6 * way[k] for k, v in b.a.items()}, 1e-6, 0.5) for s in (1, -1))
    slope = float((((up[0] - down[0]) * b.dz + (up[1] - down[1]) * b.dn) / 2e-6).sum())
    terms = [want[k].double().cpu() * way[k] for k in there]
    assert abs(sum(float(t.sum()) for t in terms) - slope) <= 200 * E * sum(float(t.abs().sum()) for t in terms) + 1e-6 * abs(slope)


@pytest.mark.gpu
def test_autograd_parts():
    b = Block(12, 64)
    d = b.device()
    r = d["r"].clone().requires_grad_()
    args = (d["y"], d["w_post"], d["gate"], d["w_pre"])
    # only one of the two results is used; a gradient that repeats one element
    z, n = cbd.block_norm(r, *args, scale=0.5)
    (g,) = torch.autograd.grad(z.sum(), r)
    assert torch.equal(g, torch.ones_like(g))
    z, n, stats = cbd.block_forward(b.plan, r, *args, save=True)
    assert z.requires_grad and n.requires_grad and not stats.requires_grad
    (g,) = torch.autograd.grad(n.sum(), r, create_graph=True)
    with torch.no_grad():
        assert torch.equal(g, cbd.block_bwd(b.plan, None, torch.ones_like(n), r, args[0], stats, *args[1:])[0])
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.sum(), r)
    with pytest.raises(ValueError, match="autograd"):
        cbd.block_forward(b.plan, r, *args, z=torch.empty_like(r))
    with pytest.raises(ValueError, match="autograd"):
        cbd.block_bwd(b.plan, r, None, d["r"], args[0], stats, *args[1:])
    z = torch.zeros_like(d["r"])
    loss = (torch.ones_like(z, requires_grad=True) * z).sum()
    cbd.block_forward(b.plan, d["r"], *args, z=z)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
    import torch.autograd.forward_ad as forward

    with forward.dual_level():
        dual = forward.make_dual(d["r"], torch.ones_like(d["r"]))
        with pytest.raises((RuntimeError, NotImplementedError)):
            cbd.block_norm(dual, *args)


# ------------------------------------------------------------ refusals (CPU)

@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), 1), (dict(c=0), 1), (dict(dtype=2), 1), (dict(dtype=cbd.F32, dw_dtype=cbd.BF16), 1),
    (dict(eps=-1e-9), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(scale=float("nan")), 1),
    (dict(scale=1e39), 1), (dict(rows=2 ** 41), 2), (dict(c=16385), 2), (dict(rows=0), 0), (dict(), 0)])
def test_plan_refusals(over, status):
    kw = dict(rows=8, c=16, dtype=cbd.BF16, dw_dtype=cbd.F32, eps=1e-6, scale=1.0)
    kw.update(over)
    h = ctypes.c_void_p()
    assert cbd._lib.cbd_block_plan(ctypes.byref(cbd.BlockProblem(**kw)), ctypes.byref(h)) == status
    assert bool(h.value) == (status == 0)
    if status:
        assert cbd._lib.cbd_last_error()
    cbd._lib.cbd_block_plan_destroy(h)


def test_run_refusals():
    """Argument checks come before any launch, so made-up addresses do."""
    L, P, S, G = cbd._lib, cbd.BlockParams, cbd.BlockStrides, cbd.BlockGrads
    p = cbd.block_plan(8, 16, dw_dtype="f32")
    r, y, a, g, b, z, n, st, dz, dn, dr, dy, ws = (0x10000 * i for i in range(1, 14))

    def fwd(r=r, y=y, w=(a, g, b, 1, 0), z=z, n=n, stats=st, s=None, plan=p._h):
        return L.cbd_block_forward(plan, r, y, ctypes.byref(P(*w)) if w else None, z, n, stats,
                                   ctypes.byref(s) if s else None, None)

    assert fwd(plan=None) == 1 and fwd(r=None) == 1
    assert fwd(y=None) == 1 and fwd(z=None) == 1 and fwd(n=None) == 1 and fwd(w=None) == 1
    assert fwd(y=None, z=None, w=(a, None, b, 0, 0)) == 1 and fwd(y=None, z=None, w=(None, g, b, 1, 0)) == 1
    assert fwd(w=(a, g, None, 1, 0)) == 1 and fwd(w=(a, g, b, 0, 0)) == 1 and fwd(w=(a, None, b, 1, 0)) == 1
    assert fwd(w=(a, None, b, 2, 0)) == 1 and fwd(w=(a, g, b, 3, 0)) == 1 and fwd(w=(a, g, b, 1, 1)) == 1
    for k in ("r", "y", "z", "n"):
        assert fwd(**{k: dict(r=r, y=y, z=z, n=n)[k] + 1}) == 2
    assert fwd(stats=st + 2) == 2 and fwd(w=(a + 1, g, b, 1, 0)) == 2
    assert fwd(z=y) == 1 and fwd(n=r) == 1 and fwd(z=n) == 1 and fwd(z=r + 2) == 1 and fwd(n=b) == 1
    assert fwd(z=r, s=S(r=20, z=24)) == 1 and fwd(stats=y) == 1
    assert fwd(s=S(r=15)) == 1 and fwd(s=S(n=-1)) == 1 and fwd(s=S(y=2 ** 31 + 1)) == 2

    def bwd(dz=dz, dn=dn, r=r, y=y, stats=st, w=(a, g, b, 1, 0), grads=(dr, dy, z, n, n + 64), s=None, ws=ws, size=1 << 20,
            plan=p._h):
        return L.cbd_block_bwd(plan, dz, dn, r, y, stats, ctypes.byref(P(*w)), ctypes.byref(G(*grads)) if grads else None,
                               ctypes.byref(s) if s else None, ws, size, None)

    assert bwd(plan=None) == 1 and bwd(r=None) == 1 and bwd(stats=None) == 1 and bwd(grads=None) == 1
    assert bwd(ws=None) == 1 and bwd(size=p.workspace_size() - 1) == 1 and bwd(ws=ws + 16) == 2
    assert bwd(y=None) == 1 and bwd(y=None, w=(None, None, b, 0, 0), grads=(dr, dy, None, None, n)) == 1
    assert bwd(w=(None, g, b, 1, 0)) == 1 and bwd(w=(a, None, b, 0, 0)) == 1 and bwd(w=(a, g, None, 1, 0)) == 1
    assert bwd(w=(a, g, None, 1, 0), grads=(dr, dy, z, n, None)) == 1  # dn without w_pre
    assert bwd(dz=dz + 1) == 2 and bwd(grads=(dr + 1, dy, z, n, n + 64)) == 2 and bwd(grads=(dr, dy, z + 2, n, n + 64)) == 2
    assert bwd(grads=(r, dy, z, n, n + 64)) == 1 and bwd(grads=(dr, y, z, n, n + 64)) == 1
    assert bwd(grads=(dn, dy, z, n, n + 64)) == 1 and bwd(grads=(dz + 2, dy, z, n, n + 64)) == 1
    assert bwd(grads=(dr, dr, z, n, n + 64)) == 1 and bwd(grads=(dr, dy, ws + 8, n, n + 64)) == 1
    assert bwd(grads=(dr, dy, z, z + 4, n)) == 1 and bwd(grads=(dr, dy, st, n, n + 64)) == 1
    assert bwd(s=S(dr=15)) == 1 and bwd(s=S(dgate=2 ** 40)) == 2
    none = cbd.block_plan(0, 16)
    assert fwd(plan=none._h, r=None, y=None, z=None, n=None, stats=None, w=(None, None, None, 0, 0)) == 0


def test_python_refusals_without_a_gpu():
    p = cbd.block_plan(4, 8)
    r, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        cbd.block_forward(p, r, w_pre=w)
    with pytest.raises(ValueError, match="GPU"):
        cbd.block_bwd(p, r, None, r)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        cbd.block_norm(r.half(), w_pre=w)
    with pytest.raises(ValueError, match="shape"):
        cbd.block_norm(r, r[:2], w_pre=w)


def test_operands_on_the_host_are_refused_with_gradients_too():
    p = cbd.block_plan(4, 8)
    r, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.bfloat16)
    for a, b in ((r.clone().requires_grad_(), w), (r, w.clone().requires_grad_())):
        with pytest.raises(ValueError, match="GPU"):
            cbd.block_forward(p, a, w_pre=b)
        with pytest.raises(ValueError, match="GPU"):
            cbd.block_norm(a, w_pre=b)


@pytest.mark.gpu
def test_python_refusals():
    p = cbd.block_plan(4, 8)
    g = dict(dtype=torch.bfloat16, device="cuda")
    r, y, w = torch.zeros(4, 8, **g), torch.zeros(4, 8, **g), torch.zeros(8, **g)
    for bad in (dict(r=r.float()), dict(r=r[:3]), dict(y=y[:1].expand(4, 8)), dict(y=y.cpu()), dict(w_post=w.float()),
                dict(w_post=w[:7]), dict(gate=w.cpu()), dict(gate=y[:2]), dict(w_pre=torch.zeros(16, **g)[::2]),
                dict(y=None), dict(stats=torch.zeros(4, 2, **g)), dict(z=torch.zeros(4, 9, **g))):
        kw = dict(r=r, y=y, w_post=w, gate=w, w_pre=w)
        kw.update(bad)
        with pytest.raises(ValueError):
            cbd.block_forward(p, **kw)
    with pytest.raises(ValueError, match="stats"):
        cbd.block_bwd(p, y, None, r, y, None, w)
    with pytest.raises(ValueError, match="dgate"):
        cbd.block_bwd(p, y, None, r, y, torch.ones(4, 2, device="cuda"), w, w, dgate=torch.zeros(4, 8, **g))
