"""The training example: every operator together, and the layer learns."""
from __future__ import annotations

import importlib.util
import os

import pytest


@pytest.mark.gpu
def test_layer_of_experts_learns():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_experts.py")
    spec = importlib.util.spec_from_file_location("train_experts", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, norms, dx = m.train(tokens=2048, experts=8, c=128, k=96, steps=30)
    # x has unit variance and the target rows unit norm: the first loss is
    # near 1, and a step of plain descent takes it down.
    assert 0.8 < losses[0] < 1.2 and losses[-1] < 0.5 * losses[0]
    assert all(n > 0 for n in norms) and tuple(dx.shape) == (2048, 128)
