"""A residual MLP trained on one GPU with the library's training step: fused linear maps
forward and backward, clipping by the global norm, and AdamW with 8-bit moments.

    python examples/train_mlp.py [--steps 60] [--moments 8|32]

The task is synthetic (a fixed random map to be learnt); the loss printed every ten steps
falls.  Everything runs on PyTorch's current stream.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from zero_partitioned_mixed_adam_gb300 import check_device  # noqa: E402
from zero_partitioned_mixed_adam_gb300.nn import linear  # noqa: E402
from zero_partitioned_mixed_adam_gb300.optim import TensorAdamW  # noqa: E402


def block(x, p):
    """x + W2 gelu(W1 x + b1) + b2, the sum and the activation in the maps' epilogues."""
    return linear(linear(x, p["w1"], p["b1"], act="gelu"), p["w2"], p["b2"], residual=x)


def parameters(width, hidden, layers, generator):
    def normal(*shape):
        t = torch.randn(*shape, device="cuda", generator=generator) * shape[-1] ** -0.5
        return t.bfloat16().requires_grad_()

    def zeros(n):
        return torch.zeros(n, dtype=torch.bfloat16, device="cuda", requires_grad=True)

    return [{"w1": normal(hidden, width), "b1": zeros(hidden), "w2": normal(width, hidden),
             "b2": zeros(width)} for _ in range(layers)]


def train(steps=60, width=256, hidden=1024, layers=2, tokens=1024, eight_bit=True, lr=2e-3, report=None):
    """The losses of every tenth step (and the last)."""
    gen = torch.Generator("cuda").manual_seed(0)
    net = parameters(width, hidden, layers, gen)
    flat = [t for p in net for t in p.values()]
    opt = TensorAdamW(flat, lr=lr, betas=(0.9, 0.95), weight_decay=0.01, max_norm=1.0,
                      eight_bit=eight_bit, seed=1)
    target = torch.randn(width, width, device="cuda", generator=gen).bfloat16() * width ** -0.5
    losses = []
    for step in range(1, steps + 1):
        x = torch.randn(tokens, width, device="cuda", generator=gen).bfloat16()
        y = x
        for p in net:
            y = block(y, p)
        loss = (y.float() - (x @ target).float()).square().mean()
        for t in flat:
            t.grad = None
        loss.backward()
        opt.step()
        if step % 10 == 0 or step in (1, steps):
            losses.append(loss.item())
            if report:
                report(f"step {step:4d}  loss {losses[-1]:.4f}  gradient norm {opt.norm[0].item():.3f}")
    check_device("train")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--moments", type=int, choices=(8, 32), default=8)
    a = ap.parse_args()
    train(a.steps, eight_bit=a.moments == 8, report=print)
