"""A small language model without attention trained on one GPU with the library's operators from
end to end: embedding, block norms with a learned gate, fused linear maps, softmax cross entropy
over the vocabulary against a tied table, clipping by the global norm, and AdamW.

    python examples/train_lm.py [--steps 100] [--moments 8|32]

The task is synthetic: each token is followed by a fixed other one, most of the time.
Everything runs on PyTorch's current stream.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from zero_partitioned_mixed_adam_gb300 import check_device  # noqa: E402
from zero_partitioned_mixed_adam_gb300.nn import block_norm, embedding, linear, linear_cross_entropy  # noqa: E402
from zero_partitioned_mixed_adam_gb300.optim import TensorAdamW  # noqa: E402


def parameters(vocab, width, hidden, layers, generator):
    def normal(*shape, sigma):
        return (torch.randn(*shape, device="cuda", generator=generator) * sigma).bfloat16().requires_grad_()

    def full(n, value):
        return torch.full((n,), value, dtype=torch.bfloat16, device="cuda", requires_grad=True)

    blocks = [{"norm": full(width, 1.0), "w1": normal(hidden, width, sigma=width ** -0.5), "b1": full(hidden, 0.0),
               "w2": normal(width, hidden, sigma=hidden ** -0.5), "after": full(width, 1.0), "gate": full(width, 0.5)}
              for _ in range(layers)]
    return {"table": normal(vocab, width, sigma=width ** -0.5), "blocks": blocks, "norm": full(width, 1.0)}


def tensors(net):
    return [net["table"], *(t for p in net["blocks"] for t in p.values()), net["norm"]]


def loss_of(net, ids, targets, alpha):
    """The mean cross entropy of the next tokens; targets of -100 do not count."""
    table, blocks = net["table"], net["blocks"]
    s = embedding(ids, table, scale=table.shape[1] ** 0.5)
    norms = [p["norm"] for p in blocks] + [net["norm"]]
    s, y = block_norm(s, norms[0])
    for p, norm in zip(blocks, norms[1:]):
        h = linear(linear(y, p["w1"], p["b1"], act="gelu"), p["w2"])
        # the norm after this block, its gate, the sum, and the norm before the next one
        s, y = block_norm(s, norm, h=h, post="rms", post_weight=p["after"], gate=p["gate"], alpha=alpha)
    return linear_cross_entropy(y, table, targets)


def train(steps=100, vocab=515, width=256, hidden=512, layers=2, tokens=1024, eight_bit=True, lr=2e-3, report=None):
    """The losses of every tenth step (and the last)."""
    gen = torch.Generator("cuda").manual_seed(0)
    net = parameters(vocab, width, hidden, layers, gen)
    flat = tensors(net)
    opt = TensorAdamW(flat, lr=lr, betas=(0.9, 0.95), weight_decay=0.01, max_norm=1.0, eight_bit=eight_bit, seed=1)
    follows = torch.randperm(vocab, device="cuda", generator=gen)
    losses = []
    for step in range(1, steps + 1):
        ids = torch.randint(0, vocab, (tokens,), device="cuda", generator=gen)
        kind = torch.rand(tokens, device="cuda", generator=gen)
        targets = torch.where(kind < 0.9, follows[ids], torch.randint(0, vocab, (tokens,), device="cuda", generator=gen))
        targets = torch.where(kind < 0.05, -100, targets)        # padding
        loss = loss_of(net, ids, targets, alpha=layers ** -0.5)
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
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--moments", type=int, choices=(8, 32), default=8)
    a = ap.parse_args()
    train(a.steps, eight_bit=a.moments == 8, report=print)
