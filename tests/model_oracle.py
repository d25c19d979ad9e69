"""Plain 64-bit statements of the embedding, the cross entropy and the block norms, for their
tests: elementary torch operations, nothing of the library."""
import torch

F64 = torch.float64


def cross_entropy(x, w, targets, ignore=-100, scale=None):
    """(losses, total, dx, dw, dz, z, c) of total = sum of c * losses."""
    x, w = x.to(F64), w.to(F64)
    keep = targets != ignore
    good = keep & (targets >= 0) & (targets < w.shape[0])
    x = torch.where(keep[:, None], x, torch.zeros_like(x))   # an ignored row's x does not count
    at = torch.where(good, targets, torch.zeros_like(targets)).long()[:, None]
    z = x @ w.t()
    # less the target's logit or the largest: 1 - p of the target loses nothing however small it is
    d = z - z.gather(1, at)
    top = d.amax(1, keepdim=True).clamp(min=0.0)
    others = (d - top).exp().scatter(1, at, 0.0)
    rest = others.sum(1, keepdim=True)
    whole = rest + (-top).exp()
    losses = torch.where(top > 0, top + whole.log(), rest.log1p())[:, 0]
    losses = torch.where(good, losses, torch.full_like(losses, float("nan")))
    losses = torch.where(keep, losses, torch.zeros_like(losses))
    c = scale.to(F64) if scale is not None else torch.ones_like(losses) / keep.sum()
    c = torch.where(good, c, torch.where(keep, torch.full_like(c, float("nan")), torch.zeros_like(c)))
    dz = others.scatter(1, at, -rest) / whole
    dz = torch.where(keep[:, None], dz * c[:, None], torch.zeros_like(dz))
    total = torch.where(keep, c * losses, torch.zeros_like(c)).sum()
    return losses, total, dz @ w, dz.t() @ x, dz, z, c


def embedding_grad(dy, ids, vocab, scale=1.0, padding=None):
    grad = torch.zeros((vocab, dy.shape[1]), dtype=F64, device=dy.device)
    good = (ids >= 0) & (ids < vocab)
    if padding is not None:
        good &= ids != padding
    return grad.index_add_(0, ids[good].long(), dy[good].to(F64)) * scale


def standardized(x, kind, eps):
    """(x standardized along its last dimension, the root)."""
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    root = (x.square().mean(-1, keepdim=True) + eps).sqrt()
    return x / root, root


def block_norm(r, h, post, w1, b1, gate, alpha, kind, w, b, eps):
    """(s, y) in 64 bits; differentiable."""
    s = r
    if h is not None:
        p = h
        if post != "none":
            p = standardized(p, post, eps)[0]
            p = p if w1 is None else p * w1
            p = p if b1 is None else p + b1
        if gate is not None:
            p = p * gate
        s = r + alpha * p
    y = standardized(s, kind, eps)[0]
    y = y if w is None else y * w
    return s, y if b is None else y + b
