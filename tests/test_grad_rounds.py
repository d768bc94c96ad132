"""The gradient norm and clipping where workgroups take more than one chunk and
a call more than one launch, against the definition in 64 bits (bounds as in
test_grads)."""
from __future__ import annotations

import pytest
import torch

import dnn_conv2d_bwd_amd as cbd

from test_grads import check_norm, check_scaled, exact_norm, make

# More than 2048 chunks of 64 KiB in one launch; two launches of more than 2048
# each and one of fewer; starts off the allocations' alignment, ends off a chunk.
LISTS = {
    "one-launch": ([40_000_003, 20_000_001, 77], ["f32", "bf16", "f32"]),
    "three-launches": ([301_001 + 7 * i for i in range(250)], ["bf16" if i % 10 == 3 else "f32" for i in range(250)]),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", LISTS)
def test_long_lists(name):
    sizes, types = LISTS[name]
    print("[grads]", name, flush=True)
    grads = make(sizes, types, shift=1, seed=5)
    want = exact_norm(grads)
    p = cbd.grad_plan(grads)
    first = cbd.grad_norm(p, grads)
    check_norm(first, want)
    assert torch.equal(first, cbd.grad_norm(p, grads))
    norm, outs = cbd.clip_grads(p, grads, 0.5 * want, out=True)
    assert torch.equal(norm, first)
    check_scaled(outs, grads, 0.5 * want, want)
    mine = [g.clone() for g in grads]
    cbd.clip_grads(p, mine, 0.5 * want)
    assert all(torch.equal(a, b) for a, b in zip(mine, outs))
