"""The expert layer (ragged products grouped by expert) against the plain
definition in 64 bits, and its refusals.

Bound of an element: the sum of n products in f32 in any order is off by at
most n * 2^-23 * sum|a||b| (one rounding of at most 2^-23 relative per
addition, products exact or rounded once), and the result's rounding adds half
a step (bf16 2^-8, f32 2^-24)."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import dnn_conv2d_bwd_amd as cbd

OPS = {"forward": cbd.FORWARD, "bwd_data": cbd.BWD_DATA, "bwd_weight": cbd.BWD_WEIGHT}
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------ definition

def bounds(ends, t):
    """[(begin, end)] of every expert: running maximum of the clamped ends."""
    out, at = [], 0
    for v in ends:
        nxt = max(at, min(max(int(v), 0), t))
        out.append((at, nxt))
        at = nxt
    return out


def as_ekc(w, lay):
    return w if lay == "ekc" else w.transpose(1, 2)


def plain(op, lay, spans, t, c, k, x=None, dy=None, w=None):
    """(result, sum of |products|, products per element) in 64 bits on the CPU."""
    def mul(a, b):
        return a @ b, a.abs() @ b.abs()

    if op == "bwd_weight":
        e = len(spans)
        r, s, n = torch.zeros(e, k, c, dtype=torch.float64), torch.zeros(e, k, c, dtype=torch.float64), 0
        for i, (lo, hi) in enumerate(spans):
            r[i], s[i] = mul(dy[lo:hi].t(), x[lo:hi])
            n = max(n, hi - lo)
        return as_ekc(r, lay), as_ekc(s, lay), n
    src, wide = (x, k) if op == "forward" else (dy, c)
    r, s = torch.zeros(t, wide, dtype=torch.float64), torch.zeros(t, wide, dtype=torch.float64)
    for i, (lo, hi) in enumerate(spans):
        we = as_ekc(w, lay)[i]
        r[lo:hi], s[lo:hi] = mul(src[lo:hi], we.t() if op == "forward" else we)
    return r, s, c if op == "forward" else k


def close(got, want, mass, n, dtype, name):
    half = torch.finfo(TORCH[dtype]).eps / 2
    slack = n * 2.0 ** -23 * mass
    tol = slack + half * (want.abs() + slack) + 1e-38
    err = (got - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol)[bad].max())} x"


# ------------------------------------------------------------ device calls

class Call:
    """One operator on the device: operands in buffers with `gap` extra
    elements a row and `off` elements before them, NaN in both, and an output
    that starts as NaN between NaN guards."""

    def __init__(self, op, lay, t, e, c, k, ends, dtype="bf16", dw="f32", gap=0, off=0, seed=0, integers=False,
                 kernel=cbd.EXPERT_KERNEL_AUTO, bits=32):
        self.op, self.lay, self.t, self.e, self.c, self.k = op, lay, t, e, c, k
        self.dtype, self.out_dtype = dtype, dw if op == "bwd_weight" else dtype
        self.gap, self.off = gap, off
        self.spans = bounds(ends, t)
        gen = torch.Generator().manual_seed(1000 + seed)

        def draw(*shape):
            if integers:
                return torch.randint(-2, 3, shape, generator=gen).float()
            return torch.randn(*shape, generator=gen).to(TORCH[dtype]).float()

        self.x, self.dy = draw(t, c), draw(t, k)
        self.w = draw(*((e, k, c) if lay == "ekc" else (e, c, k)))
        self.ends = torch.tensor(ends, dtype=torch.int32 if bits == 32 else torch.int64).cuda()
        self.plan = cbd.expert_plan(t, e, c, k, lay, dtype, dw, force_kernel=kernel)

    def view(self, shape, dtype, fill=None):
        """A device view of `shape` with the gaps; its whole buffer."""
        rows, width = int(np.prod(shape[:-1])), shape[-1]
        buf = torch.full((self.off + rows * (width + self.gap) + 64,), float("nan"), dtype=dtype, device="cuda")
        v = buf[self.off:self.off + rows * (width + self.gap)].view(rows, width + self.gap)[:, :width]
        if fill is not None:
            v.copy_(fill.reshape(rows, width).to(dtype))
        if len(shape) == 3:
            v = v.unflatten(0, (shape[0], shape[1]))
        return v, buf

    def __call__(self, accumulate=None, stream=None):
        dt, p = TORCH[self.dtype], self.plan
        x, dy, w = (self.view(tuple(v.shape), dt, v)[0] for v in (self.x, self.dy, self.w))
        shape = {"forward": (self.t, self.k), "bwd_data": (self.t, self.c), "bwd_weight": tuple(self.w.shape)}[self.op]
        out, buf = self.view(shape, TORCH[self.out_dtype], accumulate)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        if self.op == "forward":
            r = cbd.expert_forward(p, x, w, self.ends, out, stream=stream)
        elif self.op == "bwd_data":
            r = cbd.expert_bwd_data(p, dy, w, self.ends, out, stream=stream)
        else:
            r = cbd.expert_bwd_weight(p, dy, x, self.ends, out, accumulate is not None, stream=stream)
        assert r is out
        torch.cuda.synchronize()
        res = out.double().cpu()
        out.fill_(float("nan"))
        assert bool(torch.isnan(buf).all()), "a store outside the output"
        return res

    def plain(self):
        return plain(self.op, self.lay, self.spans, self.t, self.c, self.k,
                     x=self.x.double(), dy=self.dy.double(), w=self.w.double())

    def check(self):
        want, mass, n = self.plain()
        close(self(), want, mass, n, self.out_dtype, f"{self.op} {self.lay} {self.dtype}")


def split(t, e, seed, empty=0.3):
    """Random ends of e experts over t rows, some empty."""
    rng = np.random.default_rng(seed)
    w = rng.exponential(size=e) * (rng.random(e) > empty)
    if w.sum() == 0:
        w[0] = 1.0
    return np.cumsum(rng.multinomial(t, w / w.sum())).tolist()


ALL = [(op, lay) for op in OPS for lay in ("ekc", "eck")]

# rows, experts, c, k: one row; a few; tiles that end inside; experts over a wave.
SIZES = [(1, 1, 1, 1), (1, 8, 64, 64), (8, 64, 128, 96), (37, 3, 40, 72), (300, 5, 200, 136), (130, 130, 32, 48),
         (515, 2, 264, 520), (259, 64, 17, 33), (700, 7, 129, 257)]


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("op,lay", ALL)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_against_definition(dtype, op, lay, size):
    t, e, c, k = size
    print("[expert]", dtype, op, lay, size, flush=True)
    Call(op, lay, t, e, c, k, split(t, e, seed=t), dtype=dtype, seed=t).check()


@pytest.mark.gpu
@pytest.mark.parametrize("op,lay", ALL)
@pytest.mark.parametrize("gap,off", [(8, 0), (1, 0), (0, 1), (3, 5), (64, 8)])
def test_strides_and_alignment(op, lay, gap, off):
    for dtype in ("bf16", "f32"):
        print("[expert]", dtype, op, lay, gap, off, flush=True)
        Call(op, lay, 150, 4, 72, 104, split(150, 4, 3), dtype=dtype, gap=gap, off=off).check()


@pytest.mark.gpu
@pytest.mark.parametrize("op,lay", ALL)
def test_integers_are_exact(op, lay):
    for dtype in ("bf16", "f32"):
        call = Call(op, lay, 120, 6, 48, 56, split(120, 6, 9), dtype=dtype, dw=dtype, integers=True)
        want = call.plain()[0].to(TORCH[dtype]).double()
        assert torch.equal(call(), want)


ENDS = {
    "one-expert-has-all": [0, 0, 90, 90, 90],
    "none": [0, 0, 0, 0, 0],
    "rows-left-over": [3, 10, 10, 20, 41],
    "past-the-end": [30, 95, 1000, 2 ** 31 - 1, 5],
    "falling": [50, 20, 60, 10, 90],
    "negative": [-5, 30, -(2 ** 31), 60, 90],
}


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 64])
@pytest.mark.parametrize("ends", ENDS, ids=str)
@pytest.mark.parametrize("op,lay", ALL)
def test_any_ends(op, lay, ends, bits):
    """Whatever `ends` holds, rows are owned once and nothing outside is touched."""
    v = list(ENDS[ends])
    if bits == 64 and ends == "past-the-end":
        v[2] = 2 ** 62
    Call(op, lay, 90, 5, 72, 40, v, bits=bits).check()


@pytest.mark.gpu
@pytest.mark.parametrize("op,lay", ALL)
def test_no_rows(op, lay):
    call = Call(op, lay, 0, 3, 40, 24, [0, 0, 0])
    assert torch.equal(call(), call.plain()[0])


@pytest.mark.gpu
@pytest.mark.parametrize("op,lay", ALL)
def test_rows_stay_apart(op, lay):
    """NaN and infinities in one expert's rows reach no other expert's results
    (nor, for y and dx, any other row's)."""
    t, e, c, k = 200, 4, 72, 104
    ends = [45, 46, 130, 190]
    call = Call(op, lay, t, e, c, k, ends)
    clean = call()
    for v in (call.x, call.dy):
        v[45] = float("nan")      # all of expert 1
        v[130:135] = float("inf")  # expert 3's first rows
        v[195] = float("nan")     # no expert's row
    call.w[1] = float("nan")
    got = call()
    if op == "bwd_weight":
        assert torch.equal(got[[0, 2]], clean[[0, 2]])
        assert not torch.isfinite(got[1]).any() and not torch.isfinite(got[3]).any()
    else:
        keep = [i for i in range(t) if i != 45 and not 130 <= i < 135]
        assert torch.equal(got[keep], clean[keep])
        assert torch.isnan(got[45]).all() and (got[190:] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("lay", ["ekc", "eck"])
@pytest.mark.parametrize("dw", ["f32", "bf16"])
def test_accumulate(lay, dw):
    call = Call("bwd_weight", lay, 150, 5, 72, 104, [40, 40, 77, 150, 150], dw=dw)
    old = torch.randn(*call.w.shape, generator=torch.Generator().manual_seed(5)).to(TORCH[dw]).double()
    want, mass, n = call.plain()
    got = call(accumulate=old)
    # One more f32 addition and, for bf16, the one rounding of the sum.
    close(got, want + old, mass + old.abs() + want.abs(), n + 1, dw, "accumulate")
    assert torch.equal(got[1], old[1]) and torch.equal(got[4], old[4])


@pytest.mark.gpu
def test_gradients_match_differences():
    """bwd_data and bwd_weight as derivatives of sum(forward * dy): with
    small-integer operands the function is linear in each operand, so a unit
    step's difference is exact."""
    t, e, c, k = 24, 3, 16, 8
    ends = [10, 10, 22]
    f = Call("forward", "ekc", t, e, c, k, ends, dtype="f32", integers=True)
    dx = Call("bwd_data", "ekc", t, e, c, k, ends, dtype="f32", integers=True)()
    dw = Call("bwd_weight", "ekc", t, e, c, k, ends, dtype="f32", integers=True)()

    def value():
        return float((f() * f.dy.double()).sum())

    base = value()
    for r, i in [(0, 0), (9, 15), (10, 3), (21, 7), (23, 2)]:
        f.x[r, i] += 1
        assert value() - base == float(dx[r, i])
        f.x[r, i] -= 1
    for n, i, j in [(0, 0, 0), (1, 3, 4), (2, 7, 15)]:
        f.w[n, i, j] += 1
        assert value() - base == float(dw[n, i, j])
        f.w[n, i, j] -= 1


@pytest.mark.gpu
@pytest.mark.parametrize("op,lay", ALL)
def test_other_stream_and_repeats(op, lay):
    call = Call(op, lay, 300, 6, 136, 72, split(300, 6, 1))
    first = call()
    assert torch.equal(first, call(stream=torch.cuda.Stream()))
    assert torch.equal(first, call())


@pytest.mark.gpu
def test_graph_replays():
    """forward, bwd_data and bwd_weight in one captured graph, replayed with
    other values and other ends; eager work and synchronisation in between."""
    t, e, c, k = 260, 5, 136, 200
    p = cbd.expert_plan(t, e, c, k, "ekc", "bf16", "f32")
    gen = torch.Generator(device="cuda").manual_seed(3)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, dy, w = (torch.randn(*s, generator=gen, **bf) for s in ((t, c), (t, k), (e, k, c)))
    ends = torch.tensor([50, 50, 120, 200, 260], dtype=torch.int32, device="cuda")
    y, dx = torch.empty(t, k, **bf), torch.empty(t, c, **bf)
    dw = torch.empty(e, k, c, device="cuda")

    def step():
        cbd.expert_forward(p, x, w, ends, y)
        cbd.expert_bwd_data(p, dy, w, ends, dx)
        cbd.expert_bwd_weight(p, dy, x, ends, dw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        x.copy_(torch.randn(t, c, generator=gen, **bf))
        ends.copy_(torch.tensor(split(t - i, e, i), dtype=torch.int32))
        for o in (y, dx, dw):
            o.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in (y, dx, dw)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (y, dx, dw))), i


@pytest.mark.gpu
def test_fused_weights_view_and_convenience():
    """A slice of a wider weight tensor, int64 ends straight from cumsum, and
    the calls that make their own plan."""
    t, e, c, k = 96, 4, 64, 48
    gen = torch.Generator(device="cuda").manual_seed(8)
    both = torch.randint(-2, 3, (e, 2 * k, c), generator=gen, device="cuda").bfloat16()
    x = torch.randint(-2, 3, (t, c), generator=gen, device="cuda").bfloat16()
    ids = torch.randint(0, e, (t,), generator=gen, device="cuda").sort().values
    ends = torch.bincount(ids, minlength=e).cumsum(0)
    w = both[:, k:]
    y = cbd.expert_linear(x, w, ends)
    want = torch.stack([w[i].float() @ x[r].float() for r, i in enumerate(ids.tolist())]).bfloat16()
    assert torch.equal(y, want)
    dx, dw = cbd.expert_linear_bwd(y, x, w, ends, dw_dtype="f32")
    assert dx.shape == x.shape and dw.shape == w.shape and dw.dtype == torch.float32
    for i in range(e):
        rows = ids == i
        assert torch.equal(dw[i].double(), y[rows].double().t() @ x[rows].double())


# ------------------------------------------------------------ refusals (CPU)

def c_plan(**over):
    kw = dict(tokens=8, experts=2, c=16, k=24, w_layout=0, dtype=cbd.BF16, dw_dtype=cbd.F32, ends_bits=32)
    kw.update(over)
    h = ctypes.c_void_p()
    st = cbd._lib.cbd_expert_plan(ctypes.byref(cbd.ExpertProblem(**kw)), None, ctypes.byref(h))
    return st, h


@pytest.mark.parametrize("over,status", [
    (dict(tokens=-1), 1), (dict(experts=0), 1), (dict(c=0), 1), (dict(k=-3), 1), (dict(w_layout=2), 1),
    (dict(dtype=2), 1), (dict(dtype=cbd.F32, dw_dtype=cbd.BF16), 1), (dict(ends_bits=16), 1),
    (dict(experts=65537), 2), (dict(tokens=2 ** 31), 2), (dict(c=2 ** 20 + 1), 2),
    (dict(c=2 ** 16, k=2 ** 16), 2), (dict(tokens=0), 0), (dict(), 0)])
def test_plan_refusals(over, status):
    st, h = c_plan(**over)
    assert st == status
    assert bool(h.value) == (status == 0)
    if status:
        assert cbd._lib.cbd_last_error()
    cbd._lib.cbd_expert_plan_destroy(h)


def test_plan_null_and_options():
    h = ctypes.c_void_p()
    assert cbd._lib.cbd_expert_plan(None, None, ctypes.byref(h)) == 1
    with pytest.raises(cbd.CbdError):
        cbd.expert_plan(4, 2, 8, 8, force_kernel=99)
    p = cbd.expert_plan(4, 2, 8, 8)
    with pytest.raises(cbd.CbdError):
        p.info(7)
    for op in OPS.values():
        i = p.info(op)
        assert i.grid > 0 and i.flops == 2 * 4 * 8 * 8


def test_run_refusals():
    """Argument checks come before any launch, so made-up addresses do."""
    st, h = c_plan()
    assert st == 0
    L, S = cbd._lib, cbd.ExpertStrides
    x, w, ends, y = 0x10000, 0x20000, 0x30000, 0x40000

    def fwd(x=x, w=w, ends=ends, y=y, s=None, plan=h):
        return L.cbd_expert_forward(plan, x, w, ends, y, ctypes.byref(s) if s else None, None)

    assert fwd(plan=None) == 1
    assert fwd(x=None) == 1 and fwd(w=None) == 1 and fwd(ends=None) == 1 and fwd(y=None) == 1
    assert fwd(x=x + 1) == 2 and fwd(w=w + 1) == 2 and fwd(ends=ends + 2) == 2 and fwd(y=y + 1) == 2
    assert fwd(y=x) == 1 and fwd(y=x + 8 * 16 * 2 - 2) == 1 and fwd(y=w + 2) == 1 and fwd(y=ends - 2) == 1
    assert fwd(s=S(15, 0, 0, 0)) == 1 and fwd(s=S(0, 23, 0, 0)) == 1 and fwd(s=S(0, 0, 15, 0)) == 1
    assert fwd(s=S(-16, 0, 0, 0)) == 1 and fwd(s=S(0, 0, 0, 24 * 16 - 1)) == 1
    assert fwd(s=S(1 << 23, 0, 0, 0)) == 2 and fwd(s=S(0, 0, 1 << 27, 1 << 33)) == 2
    assert fwd(s=S(0, 0, 0, 1 << 41)) == 2
    # y inside x's rows, interleaved column slices that overlap by one element
    assert fwd(y=x + 15 * 2, s=S(40, 40, 0, 0)) == 1
    assert L.cbd_expert_bwd_weight(h, y, x, ends, x, 0, None, None) == 1
    assert L.cbd_expert_bwd_weight(h, y, x, ends, w, 2, None, None) == 1
    assert L.cbd_expert_bwd_weight(h, y, x, ends, w + 2, 0, None, None) == 2  # dW is f32
    L.cbd_expert_plan_destroy(h)
    # no rows: row tensors may be NULL, and nothing is launched
    st, h = c_plan(tokens=0)
    assert L.cbd_expert_forward(h, None, w, ends, None, None, None) == 0
    assert L.cbd_expert_bwd_weight(h, None, None, ends, w, 1, None, None) == 0
    assert L.cbd_expert_forward(h, None, None, ends, None, None, None) == 1
    L.cbd_expert_plan_destroy(h)


def test_python_refuses_host_tensors():
    p = cbd.expert_plan(4, 2, 8, 8)
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    w = torch.zeros(2, 8, 8, dtype=torch.bfloat16)
    ends = torch.tensor([2, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        cbd.expert_forward(p, x, w, ends)
    with pytest.raises(ValueError, match="accumulate"):
        cbd.expert_bwd_weight(p, x, x, ends, accumulate=True)


@pytest.mark.gpu
def test_python_refusals():
    p = cbd.expert_plan(4, 2, 8, 8)
    g = dict(dtype=torch.bfloat16, device="cuda")
    x, w = torch.zeros(4, 8, **g), torch.zeros(2, 8, 8, **g)
    ends = torch.tensor([2, 4], dtype=torch.int32, device="cuda")
    cbd.expert_forward(p, x, w, ends)
    for bad in (dict(x=x.float()), dict(x=x[:3]), dict(x=x.t().contiguous().t()), dict(x=x[:1].expand(4, 8)),
                dict(w=w[:1]), dict(w=w.transpose(1, 2)), dict(ends=ends[:1]), dict(ends=ends.float()),
                dict(ends=ends.cpu()), dict(y=torch.zeros(4, 9, **g))):
        kw = dict(x=x, w=w, ends=ends, y=None)
        kw.update(bad)
        with pytest.raises(ValueError):
            cbd.expert_forward(p, kw["x"], kw["w"], kw["ends"], kw["y"])
    with pytest.raises(cbd.CbdError, match="overlaps"):
        cbd.expert_forward(p, x, w, ends, x)
