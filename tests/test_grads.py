"""The global gradient norm and clipping against the definition in 64 bits,
and their refusals.

norm: squares and sums are in 64 bits, so only the rounding to f32 counts
(2^-24 relative) and the 64-bit sums' own error, below n * 2^-53.  out: the
64-bit product is rounded to f32 (2^-24) and, for bf16, once more (2^-8)."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

import dnn_conv2d_bwd_amd as cbd

TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(sizes, types, shift=0, seed=0, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, (n, t) in enumerate(zip(sizes, types)):
        off = shift * (i % 3)
        buf = torch.empty(n + off, dtype=TORCH[t], device="cuda").normal_(0.0, scale, generator=gen)
        out.append(buf[off:])
    return out


def exact_norm(grads):
    return math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads))


def check_norm(got, want):
    assert abs(float(got) - want) <= (2.0 ** -24 + 1e-12) * want


def check_scaled(outs, grads, max_norm, want):
    by = min(1.0, max_norm / (want + 1e-6))
    for o, g in zip(outs, grads):
        ref = g.double() * by
        half = torch.finfo(g.dtype).eps / 2
        tol = ref.abs() * (2.0 ** -24 + half) * (1 + 2.0 ** -20) + float(torch.finfo(g.dtype).smallest_normal) * half * 2
        assert bool(((o.double() - ref).abs() <= tol).all())


CASES = [
    ([1], ["f32"]), ([1], ["bf16"]), ([7, 0, 3], ["bf16", "f32", "f32"]),
    ([4096, 8192, 5], ["f32", "bf16", "bf16"]),
    ([16384, 16385, 32768, 32769, 65535], ["f32", "f32", "bf16", "bf16", "bf16"]),
    ([100_003, 1, 999_999, 70_001], ["bf16", "f32", "f32", "bf16"]),
    ([17 * i % 301 for i in range(250)], ["bf16" if i % 3 else "f32" for i in range(250)]),
    ([40_000_001], ["bf16"]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_norm_and_clip(case, shift):
    sizes, types = CASES[case]
    print("[grads]", case, shift, flush=True)
    grads = make(sizes, types, shift, seed=case)
    want = exact_norm(grads)
    p = cbd.grad_plan(grads)
    check_norm(cbd.grad_norm(p, grads), want)
    for max_norm in (0.5 * want, 2.0 * want, 0.0):
        norm, outs = cbd.clip_grads(p, grads, max_norm, out=True)
        check_norm(norm, want)
        check_scaled(outs, grads, max_norm, want)
        assert max_norm <= want or all(torch.equal(o, g) for o, g in zip(outs, grads))
    mine = [g.clone() for g in grads]
    norm = cbd.clip_grads(p, mine, 0.5 * want)
    check_norm(norm, want)
    assert all(torch.equal(a, b) for a, b in zip(mine, cbd.clip_grads(p, grads, 0.5 * want, out=True)[1]))


@pytest.mark.gpu
def test_nothing_outside_is_written():
    """Outputs inside NaN buffers, at every alignment of in and out."""
    for n in (1, 9, 31, 4097):
        for a in range(0, 9, 3):
            for b in range(0, 9, 2):
                for t in ("f32", "bf16"):
                    g = make([n + a], [t])[0][a:]
                    buf = torch.full((n + b + 40,), float("nan"), dtype=TORCH[t], device="cuda")
                    out = buf[b:b + n]
                    cbd.clip_grads(cbd.grad_plan([g]), [g], 0.25, out=[out])
                    check_scaled([out], [g], 0.25, exact_norm([g]))
                    out.fill_(float("nan"))
                    assert bool(torch.isnan(buf).all())


@pytest.mark.gpu
def test_extremes():
    """No overflow or underflow inside; non-finite gradients follow the formula."""
    big = torch.full((1000,), 3e38, device="cuda")
    n = cbd.grad_norm(cbd.grad_plan([big[:1]]), [big[:1]])
    check_norm(n, float(big[0].double()))
    assert float(cbd.grad_norm(cbd.grad_plan([big]), [big])) == math.inf  # sqrt(1000) * 3e38 passes f32
    norm, (out,) = cbd.clip_grads(cbd.grad_plan([big]), [big], 1.0, out=True)
    check_scaled([out], [big], 1.0, exact_norm([big]))  # the factor itself is computed in 64 bits
    tiny = torch.full((1000,), 1e-30, device="cuda")
    check_norm(cbd.grad_norm(cbd.grad_plan([tiny]), [tiny]), exact_norm([tiny]))
    for bad in (math.inf, math.nan):
        g = [torch.ones(100, device="cuda"), torch.ones(50, device="cuda", dtype=torch.bfloat16)]
        g[1][7] = bad
        norm, outs = cbd.clip_grads(cbd.grad_plan(g), g, 1.0, out=True)
        if math.isinf(bad):
            assert float(norm) == math.inf and float(outs[0].abs().sum()) == 0.0 and bool(torch.isnan(outs[1][7]))
        else:
            assert math.isnan(float(norm)) and bool(torch.isnan(outs[0]).all())


@pytest.mark.gpu
def test_empty_lists_and_layouts():
    check = cbd.grad_norm(cbd.grad_plan([]), [])
    assert float(check) == 0.0
    z = [torch.empty(0, device="cuda")]
    norm, outs = cbd.clip_grads(cbd.grad_plan(z), z, 1.0, out=True)
    assert float(norm) == 0.0 and outs[0].numel() == 0
    # dense in another order: a channels-last filter, a transposed matrix
    g = [torch.randn(8, 4, 3, 3, device="cuda").to(memory_format=torch.channels_last),
         torch.randn(20, 30, device="cuda").t()]
    want = exact_norm(g)
    norm, outs = cbd.clip_grads(cbd.grad_plan(g), g, 0.5, out=True)
    check_norm(norm, want)
    check_scaled(outs, g, 0.5, want)
    ref = [t.clone() for t in g]
    check_norm(cbd.clip_grad_norm(ref, 0.5), want)
    assert all(torch.equal(a, b) for a, b in zip(ref, outs))
    with pytest.raises(ValueError, match="dense"):
        cbd.grad_norm(cbd.grad_plan([g[1][:10]]), [g[1][:10]])
    with pytest.raises(ValueError, match="laid out"):
        cbd.clip_grads(cbd.grad_plan(g[1:]), g[1:], 0.5, out=[torch.empty(30, 20, device="cuda")])
    with pytest.raises(ValueError):
        cbd.grad_norm(cbd.grad_plan(g), g[:1])
    with pytest.raises(ValueError):
        cbd.grad_norm(cbd.grad_plan(g), [g[0], g[0]])
    with pytest.raises(cbd.CbdError, match="overlaps"):
        cbd.clip_grads(cbd.grad_plan([g[0], g[0]]), [g[0], g[0]], 1.0)


@pytest.mark.gpu
def test_streams_graphs_and_repeats():
    """The same bits on another stream, again, and from a graph replayed
    between eager work."""
    grads = make([70_001, 5, 300_000, 128], ["bf16", "f32", "f32", "bf16"], shift=1)
    p = cbd.grad_plan(grads)
    norm, outs = cbd.clip_grads(p, grads, 1.0, out=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    n2, o2 = cbd.clip_grads(p, grads, 1.0, out=True, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(norm, n2) and all(torch.equal(a, b) for a, b in zip(outs, o2))
    ws = torch.empty(p.workspace_size(), dtype=torch.uint8, device="cuda")
    gn = torch.empty((), device="cuda")
    go = [torch.empty_like(g) for g in grads]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cbd.clip_grads(p, grads, 1.0, out=go, norm=gn, workspace=ws)
    for i in range(4):
        for t in grads:
            t.mul_(1.25)
        for t in (gn, *go):
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        norm, outs = cbd.clip_grads(p, grads, 1.0, out=True)
        torch.cuda.synchronize()
        assert torch.equal(norm, gn) and all(torch.equal(a, b) for a, b in zip(outs, go)), i


# ------------------------------------------------------------ refusals (CPU)

def c_plan(counts, dtypes):
    h = ctypes.c_void_p()
    n = len(counts)
    st = cbd._lib.cbd_grad_plan((ctypes.c_int64 * max(n, 1))(*counts), (ctypes.c_int32 * max(n, 1))(*dtypes), n,
                                ctypes.byref(h))
    return st, h


@pytest.mark.parametrize("counts,dtypes,status", [
    ([], [], 0), ([0, 5], [0, 1], 0), ([-1], [0], 1), ([5], [2], 1), ([1 << 40], [0], 2), ([5], [-1], 1)])
def test_plan_refusals(counts, dtypes, status):
    st, h = c_plan(counts, dtypes)
    assert st == status and bool(h.value) == (status == 0)
    cbd._lib.cbd_grad_plan_destroy(h)


def test_run_refusals():
    """Argument checks come before any launch, so made-up addresses do."""
    L = cbd._lib
    assert L.cbd_grad_plan(None, None, 1, ctypes.byref(ctypes.c_void_p())) == 1
    assert L.cbd_grad_plan(None, None, -1, ctypes.byref(ctypes.c_void_p())) == 1
    st, h = c_plan([100, 0, 50], [0, 0, 1])
    V = ctypes.c_void_p * 3
    size = ctypes.c_uint64()
    assert L.cbd_grad_workspace_size(h, ctypes.byref(size)) == 0 and size.value % 256 == 0
    assert L.cbd_grad_workspace_size(h, None) == 1
    ok = V(0x10000, None, 0x20000)
    norm, ws, n = 0x30000, 0x40000, size.value

    def clip(g=ok, o=None, m=1.0, norm=norm, ws=ws, n=n, plan=h):
        return L.cbd_grad_clip(plan, g, o, m, norm, ws, n, None)

    assert clip(plan=None) == 1 and clip(g=None) == 1 and clip(norm=None) == 1 and clip(ws=None) == 1
    assert clip(n=n - 1) == 1 and clip(ws=ws + 64) == 2 and clip(norm=norm + 2) == 2
    assert clip(m=-1.0) == 1 and clip(m=float("nan")) == 1
    assert clip(g=V(0x10002, None, 0x20000)) == 2 and clip(g=V(0x10000, None, 0x20001)) == 2
    assert clip(g=V(None, None, 0x20000)) == 1
    assert clip(g=V(0x10000, None, 0x10000)) == 1                      # two tensors, one place
    assert clip(o=V(0x10004, None, 0x20000)) == 1                      # shifted onto itself
    assert clip(o=V(0x50000, None, 0x50000)) == 1                      # outputs on each other
    assert clip(o=V(0x20000, None, 0x60000)) == 1                      # an output on another gradient
    assert clip(norm=0x10004) == 1 and clip(ws=0x10100) == 1 and clip(ws=0x30000) == 1
    assert L.cbd_grad_norm(h, ok, 0x20000, ws, n, None) == 1
    L.cbd_grad_plan_destroy(h)


def test_python_refuses_host_tensors():
    g = [torch.zeros(4)]
    with pytest.raises(ValueError, match="GPU"):
        cbd.grad_norm(cbd.grad_plan(g), g)
    with pytest.raises(ValueError, match="float32 and bfloat16"):
        cbd.grad_plan([torch.zeros(4, dtype=torch.float16)])


@pytest.mark.gpu
@pytest.mark.parametrize("total", [1000, 30_000, 33_000, 130_000, 132_000, 300_000])
def test_around_one_workgroup(total):
    """Sizes around which one workgroup does the whole list."""
    for n in (1, 12, 16, 17):
        grads = make([total // n] * n, ["bf16" if i % 4 == 3 else "f32" for i in range(n)], shift=1, seed=n)
        want = exact_norm(grads)
        p = cbd.grad_plan(grads)
        check_norm(cbd.grad_norm(p, grads), want)
        norm, outs = cbd.clip_grads(p, grads, 0.5 * want, out=True)
        check_norm(norm, want)
        check_scaled(outs, grads, 0.5 * want, want)
        mine = [g.clone() for g in grads]
        cbd.clip_grads(p, mine, 0.5 * want)
        assert all(torch.equal(a, b) for a, b in zip(mine, outs))
