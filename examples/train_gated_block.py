"""Trains one residual block of gated experts on one GPU: a norm, the experts, a
norm with a gate and the residual, clipped gradients and orthogonalised updates.

    python examples/train_gated_block.py --steps 40

Tokens of a mixture are sorted by their expert; the block has to learn another
block's map of them.  Weights are kept in f32 and used in bf16; matrices are
updated by their orthogonalised momentum, vectors by their clipped gradient.
Nothing in a step waits for the GPU.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dnn_conv2d_bwd_amd as cbd  # noqa: E402

MATRICES = ("w", "down")  # [E, 2K, C] and [E, C, K]; the others are vectors of C


def init(experts, c, k, gen, scale=1.0):
    """A block's parameters, in f32."""
    def normal(*shape, by):
        return by * torch.randn(*shape, generator=gen, device="cuda")

    return dict(w=normal(experts, 2 * k, c, by=scale * c ** -0.5), down=normal(experts, c, k, by=scale * k ** -0.5),
                w_pre=1.0 + normal(c, by=0.1), w_post=1.0 + normal(c, by=0.1), gate=normal(c, by=0.5))


def forward(p, r, ends):
    """The residual stream after the block, and what the next one would read."""
    _, n = cbd.block_norm(r, w_pre=p["w_pre"])
    y = cbd.expert_ffn(n, p["w"], p["down"], ends)
    return cbd.block_norm(r, y, p["w_post"], p["gate"], p["w_pre"], scale=0.5)


def route(tokens, experts, gen):
    """A router's choice: an expert per token, and the tokens in its order."""
    choice = torch.randint(0, experts, (tokens,), generator=gen, device="cuda")
    return choice.argsort(stable=True), torch.bincount(choice, minlength=experts).cumsum(0)


def train(tokens=4096, experts=16, c=512, k=256, steps=40, seed=0, rate=0.02, momentum=0.9, max_norm=1.0):
    """The losses, the gradient norms and the last step's gradient of the tokens."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    target = {n: t.bfloat16() for n, t in init(experts, c, k, gen).items()}
    param = init(experts, c, k, gen, scale=0.5)
    memory = {n: torch.zeros_like(param[n]) for n in MATRICES}
    plans = {n: cbd.ortho_plan(*param[n].shape, dtype="f32", scale=0.2) for n in MATRICES}
    names = list(param)
    clipping = None
    losses, norms = [], []
    for _ in range(steps):
        r = torch.randn(tokens, c, generator=gen, device="cuda").bfloat16()
        order, ends = route(tokens, experts, gen)
        r = r[order]
        with torch.no_grad():
            want, _ = forward(target, r, ends)
        leaf = {n: t.bfloat16().requires_grad_() for n, t in param.items()}
        r.requires_grad_()
        z, _ = forward(leaf, r, ends)
        loss = (z.float() - want.float()).square().mean()
        *grads, dr = torch.autograd.grad(loss, [leaf[n] for n in names] + [r])
        clipping = clipping or cbd.grad_plan(grads)
        norms.append(cbd.clip_grads(clipping, grads, max_norm))
        losses.append(loss.detach())
        for n, g in zip(names, grads):
            if n in MATRICES:
                memory[n].mul_(momentum).add_(g)
                param[n].sub_(rate * cbd.orthogonalize(plans[n], memory[n]))
            else:
                param[n].sub_(rate * c * g)
    return torch.stack(losses).tolist(), torch.stack(norms).tolist(), dr


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--experts", type=int, default=16)
    a = ap.parse_args()
    losses, norms, dr = train(tokens=a.tokens, experts=a.experts, steps=a.steps)
    for i in sorted({*range(0, a.steps, max(1, a.steps // 8)), a.steps - 1}):
        print(f"step {i:4d}  loss {losses[i]:.4f}  gradient norm {norms[i]:.4f}")
    print(f"gradient of the tokens: {tuple(dr.shape)}, {dr.dtype}")


if __name__ == "__main__":
    main()
