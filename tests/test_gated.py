"""Gated experts against the plain definition in 64 bits, their refusals, and
the differentiable block.

Bounds.  With n products an f32 sum is off by at most d = n * 2^-23 * sum|a||b|
(test_experts).  The step s(g) = 1 / (1 + exp(-t)) is computed with exp's
argument, exp and the reciprocal each off by a few units of 2^-23, the argument
by |t| of them: s is off by at most (|t| + 8) * 2^-22 of itself.  act(g) = g s
has a slope of at most 1.13 in g.  The derivative s + s (1 - s) g t', of a g that
is given exactly, is off by the step's error times 1 + |g t'| at most.  Results
add half a step (bf16 2^-8, f32 2^-24)."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

import dnn_conv2d_bwd_amd as cbd

from test_experts import ENDS, TORCH, as_ekc, bounds, split

GELU = math.sqrt(2.0 / math.pi)
ACTS = ("silu", "gelu", "relu")


# ------------------------------------------------------------ definition

def step(act, g):
    """s(g), t(g) and t'(g) in 64 bits."""
    if act == "relu":
        return (g > 0).to(g.dtype), torch.zeros_like(g), torch.zeros_like(g)
    t = g if act == "silu" else 2 * GELU * (g + 0.044715 * g ** 3)
    dt = torch.ones_like(g) if act == "silu" else 2 * GELU * (1 + 0.134145 * g ** 2)
    return torch.sigmoid(t), t, dt


def plain_act(act, g):
    """act, its derivative, the relative error of the step they share, and what
    the derivative multiplies it by."""
    s, t, dt = step(act, g)
    value = torch.where(g > 0, g, torch.zeros_like(g)) if act == "relu" else g * s
    # Where g is NaN it stays so.
    value = torch.where(torch.isnan(g), g, value)
    return value, s + s * (1 - s) * g * dt, (t.abs() + 8) * 2.0 ** -22, 1 + (g * dt).abs()


def products(rows, w, spans, wide):
    """rows[t] @ w[e] in 64 bits and the sums of |products|."""
    r = torch.zeros(rows.shape[0], wide, dtype=torch.float64)
    s = torch.zeros_like(r)
    for i, (lo, hi) in enumerate(spans):
        r[lo:hi], s[lo:hi] = rows[lo:hi] @ w[i], rows[lo:hi].abs() @ w[i].abs()
    return r, s


def within(got, want, slack, dtype, name):
    tol = slack + torch.finfo(TORCH[dtype]).eps / 2 * (want.abs() + slack) + 1e-37
    err = (got - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol)[bad].max())} x"


# ------------------------------------------------------------ device calls

class Gated:
    """Both operators of one block on the device: operands in buffers with
    `gap` extra elements a row and `off` before them, NaN in both, and outputs
    that start as NaN between NaN guards."""

    def __init__(self, lay, t, e, c, k, ends, dtype="bf16", act="silu", gap=0, off=0, seed=0,
                 kernel=cbd.EXPERT_KERNEL_AUTO, bits=32):
        self.lay, self.t, self.e, self.c, self.k = lay, t, e, c, k
        self.dtype, self.act, self.gap, self.off = dtype, act, gap, off
        self.spans = bounds(ends, t)
        gen = torch.Generator().manual_seed(2000 + seed)

        def draw(*shape, scale=1.0):
            return (scale * torch.randn(*shape, generator=gen)).to(TORCH[dtype]).double()

        self.x, self.dy, self.gu = draw(t, c), draw(t, c), draw(t, 2 * k, scale=2.0)
        self.w = draw(*((e, 2 * k, c) if lay == "ekc" else (e, c, 2 * k)), scale=c ** -0.5)
        self.down = draw(*((e, c, k) if lay == "ekc" else (e, k, c)), scale=k ** -0.5)
        self.ends = torch.tensor(ends, dtype=torch.int32 if bits == 32 else torch.int64).cuda()
        self.p = cbd.expert_plan(t, e, c, 2 * k, lay, dtype, force_kernel=kernel)
        self.d = cbd.expert_plan(t, e, k, c, lay, dtype, force_kernel=kernel)

    def view(self, shape, fill=None):
        rows, width = math.prod(shape[:-1]), shape[-1]
        n = self.off + rows * (width + self.gap)
        buf = torch.full((n + 64,), float("nan"), dtype=TORCH[self.dtype], device="cuda")
        v = buf[self.off:n].view(rows, width + self.gap)[:, :width]
        if fill is not None:
            v.copy_(fill.reshape(rows, width).to(TORCH[self.dtype]))
        return (v.unflatten(0, shape[:2]) if len(shape) == 3 else v), buf

    def read(self, out, buf):
        torch.cuda.synchronize()
        res = out.double().cpu()
        out.fill_(float("nan"))
        assert bool(torch.isnan(buf).all()), "a store outside the output"
        return res

    def forward(self, save, stream=None):
        x, w = self.view(tuple(self.x.shape), self.x)[0], self.view(tuple(self.w.shape), self.w)[0]
        h, hb = self.view((self.t, self.k))
        gu, gb = self.view((self.t, 2 * self.k)) if save else (None, None)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        r = cbd.expert_gated_forward(self.p, x, w, self.ends, self.act, h=h, gu=gu, stream=stream)
        if not save:
            assert r is h
            return self.read(h, hb), None
        assert r[0] is h and r[1] is gu
        return self.read(h, hb), self.read(gu, gb)

    def bwd(self, stream=None):
        dy, w, gu = (self.view(tuple(v.shape), v)[0] for v in (self.dy, self.down, self.gu))
        dgu, buf = self.view((self.t, 2 * self.k))
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        assert cbd.expert_gated_bwd(self.d, dy, w, gu, self.ends, self.act, dgu, stream=stream) is dgu
        return self.read(dgu, buf)

    def check(self, saves=(False, True), bwd=True):
        k, name = self.k, f"{self.lay} {self.dtype} {self.act}"
        both, mass = products(self.x, as_ekc(self.w, self.lay).transpose(1, 2), self.spans, 2 * k)
        d = self.c * 2.0 ** -23 * mass
        (g, u), (dg, du) = both.split(k, 1), d.split(k, 1)
        a, _, off, _ = plain_act(self.act, g)
        # act within [g - dg, g + dg], times u within its own.
        da = 1.13 * dg + off * a.abs()
        for save in saves:
            h, gu = self.forward(save)
            within(h, a * u, da * (u.abs() + du) + a.abs() * du + off * (a * u).abs(), self.dtype, name + " h")
            if save:
                within(gu, both, d, self.dtype, name + " gu")
        if bwd:
            dh, mass = products(self.dy, as_ekc(self.down, self.lay), self.spans, k)
            d = self.c * 2.0 ** -23 * mass
            g, u = self.gu.split(k, 1)
            a, slope, off, more = plain_act(self.act, g)
            want = torch.cat([dh * u * slope, dh * a], 1)
            ds = off * more * step(self.act, g)[0] + 2.0 ** -22 * slope.abs()
            slack = torch.cat([u.abs() * (d * slope.abs() + (dh.abs() + d) * ds),
                               d * a.abs() + (dh.abs() + d) * off * a.abs()], 1) + 2.0 ** -22 * want.abs()
            within(self.bwd(), want, slack, self.dtype, name + " dgu")


LAYS = ["ekc", "eck"]
# rows, experts, c, k: one row; a few; tiles that end inside; experts over a wave.
SIZES = [(1, 1, 1, 1), (1, 8, 64, 64), (8, 64, 128, 96), (37, 3, 40, 72), (300, 5, 200, 136), (130, 130, 32, 48),
         (515, 2, 264, 260), (259, 64, 17, 33), (700, 7, 129, 127), (64, 2, 72, 3)]


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("lay", LAYS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_against_definition(dtype, lay, size):
    t, e, c, k = size
    print("[gated]", dtype, lay, size, flush=True)
    Gated(lay, t, e, c, k, split(t, e, seed=t), dtype=dtype, seed=t, act=ACTS[(t + c) % 3]).check()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [640, 3305, 4096])
@pytest.mark.parametrize("lay", LAYS)
def test_long_f32_sums(lay, n):
    """1 and n - 1 terms of 2^-25, which one sum from the front would lose (n 2^-25
    of 1).  In sums of 128 terms, the last of up to 255, that are joined, a term
    is in at most 255 + n / 128 + 2 additions, each off by at most 2^-24 of what
    it adds up to."""
    print("[gated] long sums", lay, n, flush=True)
    terms = torch.full((n,), 2.0 ** -25)
    terms[0] = 1.0
    want = 1.0 + (n - 1) * 2.0 ** -25
    tol = (255 + n / 128 + 2) * 2.0 ** -24 * want
    assert tol < (n - 1) * 2.0 ** -25 or n < 1000
    t, k, ends = 40, 24, torch.tensor([40], dtype=torch.int32, device="cuda")
    ones, w = torch.ones(t, n, device="cuda"), terms.cuda().expand(1, 2 * k, n).contiguous()
    h, gu = cbd.expert_gated_forward(cbd.expert_plan(t, 1, n, 2 * k, lay, "f32"), ones,
                                     w if lay == "ekc" else w.transpose(1, 2).contiguous(), ends, act="relu", save=True)
    assert float((gu.double() - want).abs().max()) <= tol
    assert float((h.double() - want * want).abs().max()) <= 2.0 ** -24 * want * want + 2.1 * tol
    down = w[:, :k]
    dgu = cbd.expert_gated_bwd(cbd.expert_plan(t, 1, k, n, lay, "f32"), ones,
                               down.transpose(1, 2).contiguous() if lay == "ekc" else down.contiguous(),
                               torch.ones_like(gu), ends, act="relu")
    assert float((dgu.double() - want).abs().max()) <= tol


@pytest.mark.gpu
@pytest.mark.parametrize("k", [1, 2, 3])
@pytest.mark.parametrize("n", [640, 3305, 4096])
@pytest.mark.parametrize("lay", LAYS)
def test_long_f32_sums_of_few_features(lay, n, k):
    """As test_long_f32_sums, with fewer features than a vector holds; one sum
    from the front would be off by most of what the small terms add up to."""
    print("[gated] long sums", lay, n, k, flush=True)
    terms = torch.full((n,), 2.0 ** -25)
    terms[0] = 1.0
    want = 1.0 + (n - 1) * 2.0 ** -25
    tol = (255 + n / 128 + 2) * 2.0 ** -24 * want
    t, ends = 40, torch.tensor([40], dtype=torch.int32, device="cuda")
    ones, w = torch.ones(t, n, device="cuda"), terms.cuda().expand(1, 2 * k, n).contiguous()
    h, gu = cbd.expert_gated_forward(cbd.expert_plan(t, 1, n, 2 * k, lay, "f32"), ones,
                                     w if lay == "ekc" else w.transpose(1, 2).contiguous(), ends, act="relu", save=True)
    down = w[:, :k]
    dgu = cbd.expert_gated_bwd(cbd.expert_plan(t, 1, k, n, lay, "f32"), ones,
                               down.transpose(1, 2).contiguous() if lay == "ekc" else down.contiguous(),
                               torch.ones_like(gu), ends, act="relu")
    off = [float((v.double() - want).abs().max()) for v in (gu, dgu)]
    assert max(off) <= tol, f"{off} off, {tol} allowed"
    assert float((h.double() - want * want).abs().max()) <= 2.0 ** -24 * want * want + 2.1 * tol


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("lay", LAYS)
def test_activations(lay, act):
    for dtype in ("bf16", "f32"):
        print("[gated]", lay, act, dtype, flush=True)
        Gated(lay, 90, 3, 64, 80, split(90, 3, 5), dtype=dtype, act=act).check()


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", [cbd.EXPERT_KERNEL_GENERIC, cbd.EXPERT_KERNEL_MFMA, cbd.EXPERT_KERNEL_STREAM])
@pytest.mark.parametrize("gap,off", [(0, 0), (8, 0), (1, 0), (0, 1), (3, 5), (64, 8)])
@pytest.mark.parametrize("lay", LAYS)
def test_kernels_strides_and_alignment(lay, gap, off, kernel):
    for t, c, k in ((150, 72, 104), (45, 131, 61), (33, 80, 200)):
        print("[gated]", lay, gap, off, kernel, t, c, k, flush=True)
        Gated(lay, t, 4, c, k, split(t, 4, 3), gap=gap, off=off, kernel=kernel).check()
    if kernel == cbd.EXPERT_KERNEL_GENERIC:
        Gated(lay, 150, 4, 72, 104, split(150, 4, 3), dtype="f32", gap=gap, off=off).check()


@pytest.mark.gpu
@pytest.mark.parametrize("lay", LAYS)
def test_large_tiles(lay):
    """256 x 256 tiles: more of them than compute units, experts that fill them
    in part, empty ones and rows of nobody's."""
    t, e, c, k = 9000, 5, 264, 2048
    ends = [0, 3000, 3070, 7000, 8990]
    g = Gated(lay, t, e, c, k, ends)
    assert cbd.expert_gated_info(g.p).tile_n == 256, "the rule should take the large tiles here"
    print("[gated] large", lay, flush=True)
    g.check(saves=(True,), bwd=False)
    g = Gated(lay, t, e, 264, 4096, ends)
    assert cbd.expert_gated_info(g.d, True).tile_n == 256
    print("[gated] large bwd", lay, flush=True)
    g.check(saves=())


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 64])
@pytest.mark.parametrize("ends", ENDS, ids=str)
@pytest.mark.parametrize("lay", LAYS)
def test_any_ends(lay, ends, bits):
    v = list(ENDS[ends])
    if bits == 64 and ends == "past-the-end":
        v[2] = 2 ** 62
    for kernel in (cbd.EXPERT_KERNEL_MFMA, cbd.EXPERT_KERNEL_STREAM, cbd.EXPERT_KERNEL_GENERIC):
        Gated(lay, 90, 5, 72, 40, v, bits=bits, kernel=kernel).check(bwd=kernel != cbd.EXPERT_KERNEL_STREAM)


@pytest.mark.gpu
@pytest.mark.parametrize("lay", LAYS)
def test_rows_and_experts_stay_apart(lay):
    """Infinities and NaN in one row, in one expert's weights and past the last
    expert's rows change nothing elsewhere."""
    ends = [20, 20, 50, 60]
    for kernel in (cbd.EXPERT_KERNEL_GENERIC, cbd.EXPERT_KERNEL_MFMA, cbd.EXPERT_KERNEL_STREAM):
        print("[gated] apart", lay, kernel, flush=True)
        g = Gated(lay, 64, 4, 40, 56, ends, kernel=kernel)
        h, gu = g.forward(True)
        dgu = g.bwd()
        g.x[5], g.x[61] = float("nan"), float("inf")
        g.dy[5], g.dy[61] = float("inf"), float("nan")
        g.gu[5] = float("nan")
        g.w[3], g.down[3] = float("nan"), float("inf")
        h2, gu2 = g.forward(True)
        dgu2 = g.bwd()
        same = [i for i in range(50) if i != 5]
        for a, b in ((h, h2), (gu, gu2), (dgu, dgu2)):
            assert torch.equal(a[same], b[same]) and torch.equal(a[60:], b[60:])
            assert not b[60:].any() and not torch.isfinite(b[5]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("lay", LAYS)
def test_rows_of_nobody_are_plus_zero(lay, act):
    """Whatever their operands hold, the saved projections included: NaN,
    infinities, and values whose products with 0 are -0."""
    inf, nan = float("inf"), float("nan")
    for kernel, dtype in ((cbd.EXPERT_KERNEL_GENERIC, "f32"), (cbd.EXPERT_KERNEL_GENERIC, "bf16"),
                          (cbd.EXPERT_KERNEL_MFMA, "bf16"), (cbd.EXPERT_KERNEL_STREAM, "bf16")):
        for c, k in ((40, 56), (17, 3)):
            print("[gated] nobody's", lay, act, kernel, dtype, c, k, flush=True)
            g = Gated(lay, 70, 4, c, k, [20, 20, 50, 60], dtype=dtype, act=act, kernel=kernel)
            g.x[60:], g.dy[60:], g.gu[60:] = -1.0, -1.0, -3.0
            g.x[61], g.dy[62], g.gu[63], g.gu[64], g.gu[65, 0], g.gu[66, k] = nan, inf, nan, inf, -inf, -inf
            g.gu[67, :k], g.gu[68, k:] = 2.0, 2.0
            for v in (*g.forward(True), g.forward(False)[0], g.bwd()):
                assert torch.equal(v[60:], torch.zeros_like(v[60:])) and not torch.signbit(v[60:]).any()
                assert torch.isfinite(v).all()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
def test_extreme_gates(act):
    """Far gates give what the formula's limits are, through every kernel."""
    big = [0.0, -0.0, 1e-30, 50.0, -50.0, 200.0, -200.0, 3e4, -3e4, 1e20, -1e20, 3e38, -3e38]
    c = k = 16
    for kernel in (cbd.EXPERT_KERNEL_GENERIC, cbd.EXPERT_KERNEL_MFMA, cbd.EXPERT_KERNEL_STREAM):
        for dtype in ("bf16", "f32") if kernel == cbd.EXPERT_KERNEL_GENERIC else ("bf16",):
            g = Gated("ekc", len(big), 1, c, k, [len(big)], dtype=dtype, act=act, kernel=kernel)
            # One product: g = x[0] * 1, u = x[1] * 1, so sums are exact.
            g.x.zero_()
            g.w.zero_()
            g.x[:, 0] = torch.tensor(big).to(TORCH[dtype]).double()
            g.x[:, 1] = 0.5
            g.w[0, :k, 0] = 1.0
            g.w[0, k:, 1] = 1.0
            h, gu = g.forward(True)
            value, slope, off, more = plain_act(act, g.x[:, :1].expand(-1, k))
            assert torch.equal(gu[:, :k], g.x[:, :1].expand(-1, k))
            # Below f32's normal numbers a step may be lost: |g| * 2^-126.
            lost = g.x[:, :1].abs() * 2.0 ** -125
            within(h, value * 0.5, off * value.abs() + lost, dtype, f"{act} h")
            if kernel != cbd.EXPERT_KERNEL_STREAM:
                g.gu[:, :k], g.gu[:, k:] = g.x[:, :1], 0.5
                g.dy.zero_()
                g.down.zero_()
                g.dy[:, 0], g.down[0, 0, :] = 1.0, 1.0
                dgu = g.bwd()
                step_of = step(act, g.x[:, :1].expand(-1, k))[0]
                within(dgu[:, :k], 0.5 * slope, off * more * step_of + lost * more, dtype, f"{act} dg")
                within(dgu[:, k:], value, off * value.abs() + lost, dtype, f"{act} du")


@pytest.mark.gpu
@pytest.mark.parametrize("lay", LAYS)
def test_streams_repeats_and_graph_replays(lay):
    g = Gated(lay, 100, 4, 72, 56, [30, 30, 80, 97])
    want = (*g.forward(True), g.bwd())
    s = torch.cuda.Stream()
    for stream in (None, s, s):
        got = (*g.forward(True, stream), g.bwd(stream))
        assert all(torch.equal(a, b) for a, b in zip(got, want))

    bf = torch.bfloat16
    x, w, dy, down, gu0 = (v.to(bf).cuda() for v in (g.x, g.w, g.dy, g.down, g.gu))
    ends = g.ends.clone()

    def call():
        return (*cbd.expert_gated_forward(g.p, x, w, ends, save=True), cbd.expert_gated_bwd(g.d, dy, down, gu0, ends))

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for i in range(4):
        x.mul_(0.5)
        ends.copy_(torch.tensor(split(100 - i, 4, i), dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        mine = [t.clone() for t in out]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(mine, call())), i


@pytest.mark.gpu
def test_no_rows():
    p, d = cbd.expert_plan(0, 2, 8, 8), cbd.expert_plan(0, 2, 4, 8)
    g = dict(dtype=torch.bfloat16, device="cuda")
    ends = torch.zeros(2, dtype=torch.int32, device="cuda")
    h, gu = cbd.expert_gated_forward(p, torch.empty(0, 8, **g), torch.zeros(2, 8, 8, **g), ends, save=True)
    assert h.shape == (0, 4) and gu.shape == (0, 8)
    assert cbd.expert_gated_bwd(d, torch.empty(0, 8, **g), torch.zeros(2, 8, 4, **g), gu, ends).shape == (0, 8)


# ------------------------------------------------------------ the differentiable block

def block(x, w, down, spans, act, lay):
    """The block in 64 bits."""
    w, down = as_ekc(w, lay), as_ekc(down, lay)
    out = []
    for i, (lo, hi) in enumerate(spans):
        g, u = (x[lo:hi] @ w[i].t()).chunk(2, 1)
        a = g.clamp(min=0) if act == "relu" else g * step(act, g)[0]
        out.append((a * u) @ down[i].t())
    out.append(x.new_zeros(x.shape[0] - spans[-1][1], x.shape[1]))
    return torch.cat(out)


@pytest.mark.gpu
@pytest.mark.parametrize("lay", LAYS)
@pytest.mark.parametrize("act", ACTS)
def test_block_gradients(act, lay):
    """f32 operands: the gradients are the formula's, and a directional
    difference of the device's own outputs agrees with them."""
    g = Gated(lay, 60, 3, 24, 20, [25, 25, 57], dtype="f32", act=act)
    leaves = [v.float().cuda().requires_grad_() for v in (g.x, g.w, g.down)]
    host = [v.detach().double().cpu().requires_grad_() for v in leaves]
    y = cbd.expert_ffn(*leaves, g.ends, act, lay)
    want = block(*host, g.spans, act, lay)
    dy = g.dy.float()
    got = torch.autograd.grad(y, leaves, dy.cuda())
    ref = torch.autograd.grad(want, host, dy.double())
    # Three products deep with sums of at most 60 terms, and values of order
    # one: each is off by fewer than 200 roundings of its largest terms.
    for name, a, b in zip(("y", "x", "w", "down"), (y, *got), (want, *ref)):
        scale = float(b.detach().abs().max())
        assert float((a.detach().double().cpu() - b.detach()).abs().max()) <= 200 * 2.0 ** -24 * scale, name
    # Differences, in 64 bits along a random direction: <dy, (y(+) - y(-)) / 2h>.
    gen = torch.Generator().manual_seed(1)
    way = [torch.randn(v.shape, generator=gen, dtype=torch.float64) for v in host]
    with torch.no_grad():
        step_ = 1e-6
        plus, minus = (block(*(v + s * step_ * d for v, d in zip(host, way)), g.spans, act, lay) for s in (1, -1))
        slope = float(((plus - minus) / (2 * step_) * dy.double()).sum())
    along = sum(float((a.double().cpu() * d).sum()) for a, d in zip(got, way))
    mass = sum(float((a.double().cpu() * d).abs().sum()) for a, d in zip(got, way))
    assert abs(along - slope) <= 200 * 2.0 ** -24 * mass + 1e-6 * abs(slope)


@pytest.mark.gpu
def test_block_is_its_calls():
    """bf16: outputs and gradients are, bit for bit, what the calls give; each
    gradient alone is the same; what is not needed is not kept."""
    g = Gated("ekc", 80, 4, 64, 48, [10, 30, 30, 78])
    bf = torch.bfloat16
    x, w, down, dy = (v.to(bf).cuda() for v in (g.x, g.w, g.down, g.dy))
    h, gu = cbd.expert_gated_forward(g.p, x, w, g.ends, save=True)
    y = cbd.expert_forward(g.d, h, down, g.ends)
    dgu = cbd.expert_gated_bwd(g.d, dy, down, gu, g.ends)
    want = (cbd.expert_bwd_data(g.p, dgu, w, g.ends), cbd.expert_bwd_weight(g.p, dgu, x, g.ends),
            cbd.expert_bwd_weight(g.d, dy, h, g.ends))
    for need in ((1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1)):
        leaves = [v.clone().requires_grad_(bool(n)) for v, n in zip((x, w, down), need)]
        out = cbd.expert_ffn(*leaves, g.ends)
        assert torch.equal(out, y)
        got = torch.autograd.grad(out, [v for v in leaves if v.requires_grad], dy)
        assert all(torch.equal(a, b) for a, b in zip(got, [v for v, n in zip(want, need) if n])), need
    assert not cbd.expert_ffn(x, w, down, g.ends).requires_grad
    # y.sum() hands back a gradient that repeats one element.
    v = x.clone().requires_grad_()
    cbd.expert_ffn(v, w, down, g.ends).sum().backward()
    ones = torch.ones_like(y)
    assert torch.equal(v.grad, cbd.expert_bwd_data(g.p, cbd.expert_gated_bwd(g.d, ones, down, gu, g.ends), w, g.ends))


@pytest.mark.gpu
def test_block_captured():
    """Forward and backward captured together, on leaves of the graph's own."""
    g = Gated("ekc", 80, 4, 64, 48, [10, 30, 30, 78])
    x, w, down, dy = (v.to(torch.bfloat16).cuda() for v in (g.x, g.w, g.down, g.dy))

    def step_(leaves):
        return torch.autograd.grad(cbd.expert_ffn(*leaves, g.ends), leaves, dy)

    mine = [v.requires_grad_() for v in (x, w, down)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step_(mine)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step_(mine)
    for i in range(4):
        with torch.no_grad():
            x.mul_(1.25)
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        torch.cuda.synchronize()
        other = [v.detach().clone().requires_grad_() for v in mine]
        assert all(torch.equal(a, b) for a, b in zip(kept, step_(other))), i


@pytest.mark.gpu
def test_what_autograd_cannot_record():
    g = Gated("ekc", 10, 2, 8, 8, [4, 10])
    x, w, down, dy = (v.to(torch.bfloat16).cuda() for v in (g.x, g.w, g.down, g.dy))
    with pytest.raises(ValueError, match="expert_ffn"):
        cbd.expert_gated_forward(g.p, x.clone().requires_grad_(), w, g.ends)
    with pytest.raises(ValueError, match="expert_ffn"):
        cbd.expert_gated_bwd(g.d, dy, down.clone().requires_grad_(), g.gu.to(torch.bfloat16).cuda(), g.ends)
    v = x.clone().requires_grad_()
    (first,) = torch.autograd.grad(cbd.expert_ffn(v, w, down, g.ends), v, dy, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(first.sum(), v)
    import torch.autograd.forward_ad as forward

    with forward.dual_level():
        dual = forward.make_dual(x, torch.ones_like(x))
        with pytest.raises((RuntimeError, NotImplementedError, ValueError)):
            cbd.expert_ffn(dual, w, down, g.ends)
        with pytest.raises(ValueError, match="tangent"):
            cbd.expert_gated_forward(g.p, dual, w, g.ends)


@pytest.mark.gpu
def test_written_outputs_count_as_changed():
    g = Gated("ekc", 10, 2, 8, 8, [4, 10])
    x, w, down, dy, gu = (v.to(torch.bfloat16).cuda() for v in (g.x, g.w, g.down, g.dy, g.gu))
    h, out = torch.zeros(10, 8, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(gu)
    for t, call in ((h, lambda: cbd.expert_gated_forward(g.p, x, w, g.ends, h=h)),
                    (out, lambda: cbd.expert_gated_forward(g.p, x, w, g.ends, gu=out)),
                    (out, lambda: cbd.expert_gated_bwd(g.d, dy, down, gu, g.ends, dgu=out))):
        loss = (torch.ones_like(t, requires_grad=True) * t).sum()
        call()
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()


# ------------------------------------------------------------ refusals (CPU)

def test_run_refusals():
    """Argument checks come before any launch, so made-up addresses do."""
    L, S = cbd._lib, cbd.GatedStrides
    p, d = cbd.expert_plan(8, 2, 16, 24), cbd.expert_plan(8, 2, 12, 16)
    x, w, ends, h, gu = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000

    def fwd(x=x, w=w, ends=ends, h=h, gu=gu, act=0, s=None, plan=p._h[32]):
        return L.cbd_expert_gated_forward(plan, x, w, ends, h, gu, act, ctypes.byref(s) if s else None, None)

    def bwd(dy=x, w=w, gu=gu, ends=ends, dgu=h, act=0, s=None, plan=d._h[32]):
        return L.cbd_expert_gated_bwd(plan, dy, w, gu, ends, dgu, act, ctypes.byref(s) if s else None, None)

    for f in (fwd, bwd):
        assert f(plan=None) == 1 and f(w=None) == 1 and f(ends=None) == 1
        assert f(act=3) == 1 and f(act=-1) == 1
        assert f(w=w + 1) == 2 and f(ends=ends + 2) == 2 and f(gu=gu + 1) == 2
        assert f(s=S(15, 0, 0, 0, 0, 0)) == 1 and f(s=S(0, 0, 23, 0, 0, 0)) == 1
        assert f(s=S(-16, 0, 0, 0, 0, 0)) == 1
        assert f(s=S(1 << 23, 0, 0, 0, 0, 0)) == 2 and f(s=S(0, 0, 1 << 23, 0, 0, 0)) == 2
        assert f(s=S(0, 0, 0, 0, 0, 1 << 41)) == 2 and f(s=S(0, 0, 0, 0, 1 << 27, 1 << 33)) == 2
    assert fwd(x=None) == 1 and fwd(h=None) == 1 and bwd(dy=None) == 1 and bwd(gu=None) == 1 and bwd(dgu=None) == 1
    assert fwd(x=x + 1) == 2 and fwd(h=h + 1) == 2 and bwd(dy=x + 1) == 2 and bwd(dgu=h + 1) == 2
    assert fwd(s=S(0, 11, 0, 0, 0, 0)) == 1 and bwd(s=S(0, 0, 0, 23, 0, 0)) == 1
    assert fwd(s=S(0, 0, 0, 0, 15, 0)) == 1 and bwd(s=S(0, 0, 0, 0, 11, 0)) == 1
    assert fwd(s=S(0, 1 << 23, 0, 0, 0, 0)) == 2 and bwd(s=S(0, 0, 0, 1 << 23, 0, 0)) == 2
    assert fwd(h=x) == 1 and fwd(h=w + 2) == 1 and fwd(h=ends) == 1 and fwd(h=gu + 2) == 1
    assert fwd(gu=x + 2) == 1 and fwd(gu=w) == 1 and fwd(gu=ends - 2) == 1
    assert bwd(dgu=x) == 1 and bwd(dgu=gu) == 1 and bwd(dgu=w) == 1 and bwd(dgu=ends - 2) == 1
    # An odd number of outputs cannot be two projections.
    odd = cbd.expert_plan(8, 2, 16, 23)
    assert fwd(plan=odd._h[32]) == 1
    with pytest.raises(cbd.CbdError):
        cbd.expert_gated_info(odd)
    # no rows: row tensors may be NULL, and nothing is launched
    none = cbd.expert_plan(0, 2, 16, 24)
    assert fwd(plan=none._h[32], x=None, h=None, gu=None) == 0
    assert fwd(plan=none._h[32], w=None) == 1


def test_kernel_choice():
    """Few rows an expert stream; f32 is generic; bwd never streams."""
    few, many, single = (cbd.expert_plan(t, 64, 2048, 2816) for t in (64, 65536, 1))
    assert cbd.expert_gated_info(few).kernel == cbd.EXPERT_KERNEL_STREAM == cbd.expert_gated_info(single).kernel
    assert cbd.expert_gated_info(many).kernel == cbd.EXPERT_KERNEL_MFMA
    assert cbd.expert_gated_info(cbd.expert_plan(64, 64, 2048, 1408, dtype="f32")).kernel == cbd.EXPERT_KERNEL_GENERIC
    assert cbd.expert_gated_info(cbd.expert_plan(64, 64, 1408, 2048), True).kernel == cbd.EXPERT_KERNEL_MFMA
    i = cbd.expert_gated_info(many)
    assert i.grid > 0 and i.flops == 2 * 65536 * 2048 * 2816


def test_a_forced_stream_kernel_that_does_not_take_the_call():
    """The MFMA kernel runs in its place, and the call's information says so."""
    forced = dict(force_kernel=cbd.EXPERT_KERNEL_STREAM)
    for lay in LAYS:
        p = cbd.expert_plan(4096, 4, 64, 128, lay, **forced)
        assert cbd.expert_gated_info(p).kernel == cbd.EXPERT_KERNEL_STREAM
        assert cbd.expert_gated_info(cbd.expert_plan(4096, 4, 64, 64, lay, **forced), True).kernel == cbd.EXPERT_KERNEL_MFMA
        # 2^24 workgroups or more of the stream kernel's 32 rows.
        p = cbd.expert_plan(1 << 30, 4, 8, 2, lay, **forced)
        assert cbd.expert_gated_info(p).kernel == cbd.EXPERT_KERNEL_MFMA


def test_python_refusals_without_a_gpu():
    p, d = cbd.expert_plan(4, 2, 8, 8), cbd.expert_plan(4, 2, 4, 8)
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(2, 8, 8, dtype=torch.bfloat16)
    ends = torch.tensor([2, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        cbd.expert_gated_forward(p, x, w, ends)
    with pytest.raises(ValueError, match="GPU"):
        cbd.expert_gated_bwd(d, x, w[:, :, :4], x, ends)
    with pytest.raises(ValueError, match="activation"):
        cbd.expert_gated_forward(p, x, w, ends, act="tanh")
    with pytest.raises(ValueError, match="even"):
        cbd.expert_gated_forward(cbd.expert_plan(4, 2, 8, 7), x, w[:, :7], ends)
    with pytest.raises(ValueError, match="fit"):
        cbd.expert_ffn(x, w, w, ends)
    with pytest.raises(ValueError, match="GPU"):
        cbd.expert_ffn(x, w, torch.zeros(2, 8, 4, dtype=torch.bfloat16), ends)


@pytest.mark.gpu
def test_python_refusals():
    p = cbd.expert_plan(4, 2, 8, 8)
    g = dict(dtype=torch.bfloat16, device="cuda")
    x, w = torch.zeros(4, 8, **g), torch.zeros(2, 8, 8, **g)
    ends = torch.tensor([2, 4], dtype=torch.int32, device="cuda")
    cbd.expert_gated_forward(p, x, w, ends)
    for bad in (dict(x=x.float()), dict(x=x[:3]), dict(x=x[:1].expand(4, 8)), dict(w=w[:1]),
                dict(w=w.transpose(1, 2)), dict(ends=ends[:1]), dict(ends=ends.cpu()),
                dict(h=torch.zeros(4, 5, **g)), dict(gu=torch.zeros(4, 4, **g))):
        kw = dict(x=x, w=w, ends=ends, h=None, gu=None)
        kw.update(bad)
        with pytest.raises(ValueError):
            cbd.expert_gated_forward(p, kw["x"], kw["w"], kw["ends"], h=kw["h"], gu=kw["gu"])
    both = torch.zeros(4, 12, **g)  # h and gu side by side in one buffer are fine, overlapping ones are not
    cbd.expert_gated_forward(p, x, w, ends, h=both[:, :4], gu=both[:, 4:])
    with pytest.raises(cbd.CbdError, match="overlaps"):
        cbd.expert_gated_forward(p, x, w, ends, h=both[:, 2:6], gu=both[:, 4:])
