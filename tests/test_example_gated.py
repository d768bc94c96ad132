"""The gated block's example runs, and its step's gradients are the formula's:
the norms, the experts and the residual together, as they are used, and the
clipped list and the orthogonalised updates after them."""
from __future__ import annotations

import os
import sys

import pytest
import torch

import dnn_conv2d_bwd_amd as cbd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

from test_experts import bounds  # noqa: E402


@pytest.mark.gpu
def test_example_runs():
    import train_gated_block as example

    losses, norms, dr = example.train(tokens=512, experts=4, c=64, k=48, steps=3)
    assert len(losses) == len(norms) == 3 and dr.shape == (512, 64)
    assert all(v == v and abs(v) < float("inf") for v in losses + norms) and torch.isfinite(dr).all()


def rms(v):
    return v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt()


def define(p, r, spans):
    """The example's forward pass in 64 bits."""
    n = rms(r) * p["w_pre"]
    y = []
    for i, (lo, hi) in enumerate(spans):
        g, u = (n[lo:hi] @ p["w"][i].t()).chunk(2, 1)
        y.append((g * torch.sigmoid(g) * u) @ p["down"][i].t())
    y = torch.cat(y + [r.new_zeros(r.shape[0] - spans[-1][1], r.shape[1])])
    z = r + 0.5 * p["gate"] * (p["w_post"] * rms(y))
    return z, rms(z) * p["w_pre"]


@pytest.mark.gpu
def test_step_against_definition():
    """f32 throughout.  The values are of order one and each result goes through
    two products, three norms and sums of at most 200 terms a row: fewer than 1000
    roundings of its largest terms, and a norm's row of small values raises them by
    the factor that it raises the row (y's smallest rows here: at most 10)."""
    import train_gated_block as example

    gen = torch.Generator(device="cuda").manual_seed(5)
    param = example.init(3, 64, 40, gen)
    ends = torch.tensor([50, 50, 100], device="cuda")
    r = torch.randn(100, 64, generator=gen, device="cuda")
    dz, dn = (torch.randn(100, 64, generator=gen, device="cuda") for _ in range(2))
    leaf = {n: t.clone().requires_grad_() for n, t in param.items()}
    r.requires_grad_()
    outs = example.forward(leaf, r, ends)
    got = torch.autograd.grad(outs, [*leaf.values(), r], (dz, dn))
    host = {n: t.detach().double().cpu().requires_grad_() for n, t in param.items()}
    rh = r.detach().double().cpu().requires_grad_()
    want_outs = define(host, rh, bounds(ends.tolist(), 100))
    want = torch.autograd.grad(want_outs, [*host.values(), rh], (dz.double().cpu(), dn.double().cpu()))
    for name, a, b in zip(["z", "n", *leaf, "r"], (*outs, *got), (*want_outs, *want)):
        err = float((a.detach().double().cpu() - b.detach()).abs().max())
        assert err <= 10 * 1000 * 2.0 ** -24 * float(b.detach().abs().max()), name
    # The list clipped as one, then the matrices orthogonalised: what each call says of its own.
    grads = [g.detach().clone() for g in got[:-1]]
    norm = cbd.clip_grads(cbd.grad_plan(grads), grads, 0.5)
    total = sum(float(g.double().square().sum()) for g in want[:-1]) ** 0.5
    assert abs(float(norm) - total) <= 1e-3 * total
    w = grads[list(leaf).index("w")]
    out = cbd.orthogonalized(w)
    assert torch.equal(out, cbd.orthogonalize(cbd.ortho_plan(*w.shape), w))
    # An expert without rows has no gradient, and a zero matrix no direction.
    assert not w[1].any() and not out[1].any() and torch.isfinite(out).all()
    # Five steps bring every singular value that is not tiny to between 0.6 and 1.3.
    s = torch.linalg.svdvals(out[[0, 2]].cpu())
    before = torch.linalg.svdvals(w[[0, 2]].cpu())
    big = before > 0.02 * before.norm(dim=1, keepdim=True)
    assert big.any() and ((s > 0.6) & (s < 1.3))[big].all()
