"""A plan for gradients that come from an iterator, which can be read once."""
from __future__ import annotations

import torch

import dnn_conv2d_bwd_amd as cbd


def test_plan_from_an_iterator():
    grads = [torch.zeros(5), torch.zeros(2, 3, dtype=torch.bfloat16)]
    assert cbd.grad_plan(g for g in grads).counts == cbd.grad_plan(grads).counts == (5, 6)
