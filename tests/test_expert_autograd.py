"""The expert products under autograd: what is recorded gives the gradients of
the definition, and what cannot be recorded is refused instead of detached.

On the CPU the library calls are replaced by the definition in 64 bits, so the
wiring is tested against differences; on the GPU the gradients are compared
with the calls that compute them and with the definition (bounds as in
test_experts)."""
from __future__ import annotations

import types

import pytest
import torch

import dnn_conv2d_bwd_amd as cbd
from dnn_conv2d_bwd_amd import experts

from test_experts import bounds, close, plain

T, E, C, K = 13, 4, 5, 3
ENDS = [4, 4, 9, 11]  # an expert without rows, two rows of nobody's


@pytest.fixture
def plain_calls(monkeypatch):
    """A plan for the definition in place of the library."""
    def product(p, op, rows, w, ends, out, stream):
        assert out is None
        name = ("forward", "bwd_data")[op]
        return plain(name, p.lay, bounds(ends, T), T, C, K, x=rows.detach(), dy=rows.detach(), w=w.detach())[0]

    def weight(p, dy, x, ends, dw, accumulate, stream):
        assert dw is None and not accumulate
        return plain("bwd_weight", p.lay, bounds(ends, T), T, C, K, x=x.detach(), dy=dy.detach())[0].contiguous()

    monkeypatch.setattr(experts, "_product", product)
    monkeypatch.setattr(experts, "_weight", weight)
    return lambda lay: types.SimpleNamespace(lay=lay, _tdtype=torch.float64)


def operands(lay, dtype=torch.float64, device="cpu"):
    gen = torch.Generator().manual_seed(3)

    def draw(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float64).to(dtype).to(device)

    return draw(T, C), draw(T, K), draw(*((E, K, C) if lay == "ekc" else (E, C, K)))


CALLS = {"forward": cbd.expert_forward, "bwd_data": cbd.expert_bwd_data, "bwd_weight": cbd.expert_bwd_weight}


@pytest.mark.parametrize("lay", ["ekc", "eck"])
@pytest.mark.parametrize("op", CALLS)
def test_gradients_match_differences(plain_calls, op, lay):
    """First and second derivatives, of either operand and of both."""
    p, ends = plain_calls(lay), torch.tensor(ENDS)
    x, dy, w = operands(lay)
    a, b = {"forward": (x, w), "bwd_data": (dy, w), "bwd_weight": (dy, x)}[op]
    for need_a, need_b in ((True, False), (False, True), (True, True)):
        args = a.clone().requires_grad_(need_a), b.clone().requires_grad_(need_b)
        assert torch.autograd.gradcheck(lambda u, v: CALLS[op](p, u, v, ends), args)
        assert torch.autograd.gradgradcheck(lambda u, v: CALLS[op](p, u, v, ends), args)


def test_expanded_gradients(plain_calls):
    """y.sum() hands back a gradient that repeats one element."""
    p, ends = plain_calls("ekc"), torch.tensor(ENDS)
    x, _, w = operands("ekc")
    x.requires_grad_()
    cbd.expert_forward(p, x, w, ends).sum().backward()
    want = plain("bwd_data", "ekc", bounds(ENDS, T), T, C, K, dy=torch.ones(T, K, dtype=torch.float64), w=w)[0]
    assert torch.allclose(x.grad, want)


def test_what_cannot_be_recorded_is_refused(plain_calls):
    p, ends = plain_calls("ekc"), torch.tensor(ENDS)
    x, dy, w = operands("ekc")
    w.requires_grad_()
    with pytest.raises(ValueError, match="autograd"):
        cbd.expert_forward(p, x, w, ends, torch.empty_like(dy))
    with pytest.raises(ValueError, match="autograd"):
        cbd.expert_bwd_data(p, dy, w, ends, torch.empty_like(x))
    with pytest.raises(ValueError, match="autograd"):
        cbd.expert_bwd_weight(p, dy, x.requires_grad_(), ends, torch.empty_like(w), True)
    with torch.no_grad():
        assert not cbd.expert_forward(p, x, w, ends).requires_grad
    assert cbd.expert_forward(p, x, w, ends).requires_grad
    assert not cbd.expert_forward(p, x.detach(), w.detach(), ends).requires_grad


def test_tangents_are_not_dropped(plain_calls):
    import torch.autograd.forward_ad as forward

    p, ends = plain_calls("ekc"), torch.tensor(ENDS)
    x, dy, w = operands("ekc")
    with forward.dual_level():
        dual = forward.make_dual(x, torch.ones_like(x))
        with pytest.raises((RuntimeError, NotImplementedError)):
            cbd.expert_forward(p, dual, w, ends)
        with pytest.raises(ValueError, match="tangent"):
            cbd.expert_forward(p, dual, w, ends, torch.empty_like(dy))
        assert cbd.expert_forward(p, x, w, ends).shape == dy.shape  # nothing to carry


@pytest.mark.gpu
@pytest.mark.parametrize("lay", ["ekc", "eck"])
@pytest.mark.parametrize("dtype,dw", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_against_calls_and_definition(lay, dtype, dw):
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    print("[autograd]", lay, dtype, dw, flush=True)
    x, dy, w = operands(lay, td, "cuda")
    ends = torch.tensor(ENDS, device="cuda")
    p = cbd.expert_plan(T, E, C, K, lay, dtype, dw)
    x.requires_grad_(), w.requires_grad_()
    y = cbd.expert_forward(p, x, w, ends)
    gx, gw = torch.autograd.grad(y, (x, w), dy, create_graph=True)
    with torch.no_grad():
        assert torch.equal(y, cbd.expert_forward(p, x, w, ends))
        assert torch.equal(gx, cbd.expert_bwd_data(p, dy, w, ends))
        assert torch.equal(gw, cbd.expert_bwd_weight(p, dy, x, ends).to(td))
    spans = bounds(ENDS, T)
    host = {k: v.detach().double().cpu() for k, v in dict(x=x, dy=dy, w=w).items()}
    for got, op in ((gx, "bwd_data"), (gw, "bwd_weight")):
        want, mass, n = plain(op, lay, spans, T, C, K, **host)
        # A weight gradient kept in f32 is rounded there first.
        close(got.detach().double().cpu(), want, mass, n + 1, dtype, op)
    # Second order: d/dw of <gx, v> is the weight gradient of (dy, v).
    v = torch.ones_like(x)
    (second,) = torch.autograd.grad(gx, w, v)
    with torch.no_grad():
        assert torch.equal(second, cbd.expert_bwd_weight(p, dy, v, ends).to(td))
    # and the calls that make their own plan
    z = cbd.expert_linear(x, w, ends, lay)
    assert torch.equal(torch.autograd.grad(z, x, dy)[0], gx)


@pytest.mark.gpu
def test_streams_and_graph_replays():
    """A call on a stream of its own, and forward and backward captured
    together, replayed between eager work."""
    x, dy, w = operands("ekc", torch.bfloat16, "cuda")
    ends = torch.tensor(ENDS, device="cuda")
    p = cbd.expert_plan(T, E, C, K)
    x.requires_grad_(), w.requires_grad_()

    def step(stream=None):
        return torch.autograd.grad(cbd.expert_forward(p, x, w, ends, stream=stream), (x, w), dy)

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for i in range(4):
        with torch.no_grad():
            x.mul_(1.5)
        g.replay()
        torch.cuda.synchronize()
        mine = [t.clone() for t in got]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(mine, step())), i
