"""Tensors of the caller's that the library writes to count as changed in
place: a backward pass that saved one refuses to use the new contents."""
from __future__ import annotations

import pytest
import torch

import dnn_conv2d_bwd_amd as cbd


def saved(t):
    """A loss whose backward pass needs t as it is now."""
    return (torch.ones_like(t, requires_grad=True) * t).sum()


@pytest.mark.gpu
def test_products_into_given_outputs():
    p = cbd.expert_plan(4, 2, 8, 8)
    g = dict(dtype=torch.bfloat16, device="cuda")
    x, w = torch.ones(4, 8, **g), torch.ones(2, 8, 8, **g)
    ends = torch.tensor([2, 4], dtype=torch.int32, device="cuda")
    for call, out in ((lambda o: cbd.expert_forward(p, x, w, ends, o), torch.zeros(4, 8, **g)),
                      (lambda o: cbd.expert_bwd_data(p, x, w, ends, o), torch.zeros(4, 8, **g)),
                      (lambda o: cbd.expert_bwd_weight(p, x, x, ends, o), torch.zeros(2, 8, 8, **g)),
                      (lambda o: cbd.expert_bwd_weight(p, x, x, ends, o, True), torch.zeros(2, 8, 8, **g))):
        loss = saved(out)
        call(out)
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()


@pytest.mark.gpu
def test_norm_and_clipping():
    a, b = torch.ones(100, device="cuda"), torch.ones(7, device="cuda", dtype=torch.bfloat16)
    p = cbd.grad_plan([a, b])
    for call in (lambda: cbd.clip_grads(p, [a, b], 0.5), lambda: cbd.clip_grad_norm([a, b], 0.5)):
        losses = saved(a), saved(b)
        call()
        for loss in losses:
            with pytest.raises(RuntimeError, match="inplace"):
                loss.backward()
    outs = [torch.zeros_like(a), torch.zeros_like(b)]
    norm, ws = torch.zeros((), device="cuda"), torch.empty(p.workspace_size(), dtype=torch.uint8, device="cuda")
    losses = [saved(t) for t in (*outs, norm)]
    before = a._version, ws._version
    cbd.clip_grads(p, [a, b], 0.5, out=outs, norm=norm, workspace=ws)
    assert a._version == before[0] and ws._version > before[1]  # a is only read
    for loss in losses:
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()
    loss = saved(norm)
    cbd.grad_norm(p, [a, b], norm=norm)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()


@pytest.mark.gpu
def test_inference_tensors():
    """They have no counter, and are written all the same."""
    with torch.inference_mode():
        g = [torch.full((4,), 2.0, device="cuda")]
        assert float(cbd.clip_grad_norm(g, 1.0)) == 4.0
        torch.cuda.synchronize()
        assert abs(float(g[0][0]) - 0.5) < 1e-6
