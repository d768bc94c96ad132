"""Trains a small layer of experts: forward, both gradients, clipping by the
global norm, and a plain update, on one GPU.

    python examples/train_experts.py --steps 40

Tokens of a mixture are sorted by their expert; each expert has to learn its
own linear map of them.  Weights are kept in f32 and used in bf16; gradients
stay f32 from the product to the update.  Nothing in a step waits for the GPU.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dnn_conv2d_bwd_amd as cbd  # noqa: E402


def route(tokens, experts, gen):
    """A router's choice: an expert per token, and the tokens in its order."""
    choice = torch.randint(0, experts, (tokens,), generator=gen, device="cuda")
    order = choice.argsort(stable=True)
    ends = torch.bincount(choice, minlength=experts).cumsum(0)
    return order, ends


def train(tokens=4096, experts=16, c=512, k=256, steps=40, seed=0):
    """The losses, the gradient norms and the last step's token gradients.

    The mean square's curvature is 2 / (k * experts) for a weight (an expert
    sees tokens / experts of the unit-variance rows) and 2 / k for the bias, so
    the rates below go half of the way to the minimum a step; the bound on the
    norm holds the first steps back."""
    rate, bias_rate, max_norm = 0.25 * k * experts, 0.25 * k, (k * experts) ** -0.5
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return scale * torch.randn(*shape, generator=gen, device="cuda")

    target = normal(experts, k, c, scale=c ** -0.5).bfloat16()
    weight, bias = torch.zeros(experts, k, c, device="cuda"), torch.zeros(k, device="cuda")
    products = cbd.expert_plan(tokens, experts, c, k, "ekc", "bf16", dw_dtype="f32")
    clipping = cbd.grad_plan([weight, bias])
    losses, norms = [], []
    for _ in range(steps):
        x = normal(tokens, c).bfloat16()
        order, ends = route(tokens, experts, gen)
        x = x[order]
        want = cbd.expert_forward(products, x, target, ends).float()
        w = weight.bfloat16()
        diff = cbd.expert_forward(products, x, w, ends).float() + bias - want
        losses.append(diff.square().mean())
        dy = 2.0 / diff.numel() * diff
        dw = cbd.expert_bwd_weight(products, dy.bfloat16(), x, ends)
        grads = [dw, dy.sum(0)]
        norms.append(cbd.clip_grads(clipping, grads, max_norm))
        weight -= rate * grads[0]
        bias -= bias_rate * grads[1]
    # What a layer below would train on.
    dx = cbd.expert_bwd_data(products, dy.bfloat16(), w, ends)
    return torch.stack(losses).tolist(), torch.stack(norms).tolist(), dx


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--experts", type=int, default=16)
    a = ap.parse_args()
    losses, norms, dx = train(tokens=a.tokens, experts=a.experts, steps=a.steps)
    for i in sorted({*range(0, a.steps, max(1, a.steps // 8)), a.steps - 1}):
        print(f"step {i:4d}  loss {losses[i]:.4f}  gradient norm {norms[i]:.4f}")
    print(f"gradient of the tokens: {tuple(dx.shape)}, {dx.dtype}")


if __name__ == "__main__":
    main()
