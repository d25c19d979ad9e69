"""The autograd functions of a model's ends and norms on the host: the library's calls are
replaced by 64-bit ones that take their arguments as the library does."""
import pytest
import torch

import model_oracle as o
from zero_partitioned_mixed_adam_gb300 import nn, train_ops

KINDS = {0: "none", 1: "rms", 2: "layer"}
F64 = torch.float64


def matrices(*all_):
    for t in all_:
        if t is not None and train_ops._matrix("matrix", t, *t.shape) < t.shape[1]:
            raise RuntimeError("a pitch below the width")


def lookup(ids, table, y, *, scale=1.0):
    matrices(table, y)
    assert ids.is_contiguous()
    y.copy_(table.to(F64)[ids.long()] * scale)


def scatter(dy, ids, dtable, *, scale=1.0, padding=None):
    matrices(dy, dtable)
    dtable.copy_(o.embedding_grad(dy, ids, dtable.shape[0], scale, padding))


def to64(t):
    return None if t is None else t.detach().to(F64)


def norm(r, y, *, h=None, s=None, post=0, post_weight=None, post_bias=None, gate=None, alpha=1.0, kind=1,
         weight=None, bias=None, eps=1e-5):
    matrices(r, y, h, s, gate if gate is not None and gate.dim() == 2 else None)
    out = o.block_norm(to64(r), to64(h), KINDS[post], to64(post_weight), to64(post_bias), to64(gate), alpha,
                       KINDS[kind], to64(weight), to64(bias), eps)
    if s is not None:
        s.copy_(out[0])
    y.copy_(out[1])


def norm_back(dy, s, *, ds=None, h=None, post=0, post_weight=None, post_bias=None, gate=None, alpha=1.0, kind=1,
              weight=None, eps=1e-5, dr=None, dh=None, dgate=None, dpost_weight=None, dpost_bias=None, dweight=None,
              dbias=None):
    matrices(dy, s, ds, h, dr, dh)
    with torch.enable_grad():
        at = to64(s).requires_grad_()
        w, b = (to64(t).requires_grad_() if t is not None else None for t in (weight, dbias))
        y = o.standardized(at, KINDS[kind], eps)[0]
        y = y if w is None else y * w
        (y if b is None else y + b - b.detach()).backward(to64(dy))
        d = at.grad if ds is None else at.grad + to64(ds)
        for out, leaf in ((dr, d), (dweight, w), (dbias, b)):
            if out is not None:
                out.copy_(leaf if leaf is d else leaf.grad)
        if h is None:
            return
        leaves = [to64(t).requires_grad_() if t is not None else None for t in (h, post_weight, post_bias, gate)]
        p, w1, b1, g = leaves
        if post:
            p = o.standardized(p, KINDS[post], eps)[0]
            p = p if w1 is None else p * w1
            p = p if b1 is None else p + b1
        (alpha * (p if g is None else p * g)).backward(d)
        for out, leaf in zip((dh, dpost_weight, dpost_bias, dgate), leaves):
            if out is not None:
                out.copy_(leaf.grad)


def loss(x, w, targets, losses, total, *, dx=None, dw=None, ignore_index=-100, scale=None):
    matrices(x, w, dx, dw)
    assert targets.dim() == 1 and losses is None
    ref = o.cross_entropy(x, w, targets, ignore_index, scale)
    for out, value in ((total, ref[1]), (dx, ref[2]), (dw, ref[3])):
        if out is not None:
            out.copy_(value)


@pytest.fixture(autouse=True)
def on_the_host(monkeypatch):
    for name, f in (("zero_embedding_forward", lookup), ("zero_embedding_backward", scatter),
                    ("zero_block_norm_forward", norm), ("zero_block_norm_backward", norm_back),
                    ("zero_linear_cross_entropy", loss)):
        monkeypatch.setattr(nn, name, torch.no_grad()(f))


def leaf(*shape, seed=0, sigma=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * sigma).bfloat16().requires_grad_()


def near(got, want):
    assert got.shape == want.shape and got.dtype == torch.bfloat16
    assert (got.to(F64) - want).abs().max() <= 2.0 ** -7 * want.abs().max()


@pytest.mark.parametrize("shape", [(7,), (2, 5), ()])
@pytest.mark.parametrize("padding", [None, 3])
def test_embedding(shape, padding):
    w = leaf(11, 6)
    ids = torch.randint(0, 11, shape, generator=torch.Generator().manual_seed(1))
    y = nn.embedding(ids, w, scale=2.0, padding_idx=padding)
    assert y.shape == (*shape, 6)
    dy = leaf(*shape, 6, seed=2).detach()
    y.backward(dy)
    near(w.grad, o.embedding_grad(dy.reshape(-1, 6), ids.reshape(-1), 11, 2.0, padding))
    with pytest.raises(ValueError):
        nn.embedding(ids.float(), w)


@pytest.mark.parametrize("post,gate,kind", [(None, None, "rms"), ("rms", "vector", "rms"), ("layer", "matrix", "layer")])
@pytest.mark.parametrize("use", ["both", "s", "y"])
def test_block_norm(post, gate, kind, use):
    lead, d = (3, 4), 8
    r, h = leaf(*lead, d, seed=1), leaf(*lead, d, seed=2)
    w, b = leaf(d, seed=3), leaf(d, seed=4) if kind == "layer" else None
    w1, b1 = leaf(d, seed=5) if post else None, leaf(d, seed=6) if post == "layer" else None
    g = {None: None, "vector": leaf(d, seed=7), "matrix": leaf(*lead, d, seed=7)}[gate]
    s, y = nn.block_norm(r, w, b, h=h, kind=kind, post=post, post_weight=w1, post_bias=b1, gate=g, alpha=0.5)
    ds, dy = leaf(*lead, d, seed=8).detach(), leaf(*lead, d, seed=9).detach()
    out = [(s, ds)] * (use != "y") + [(y, dy)] * (use != "s")
    torch.autograd.backward([t for t, _ in out], [t for _, t in out])
    leaves = (r, h, w1, b1, g, w, b)
    ref = [None if t is None else t.detach().to(F64).requires_grad_() for t in leaves]
    s64, y64 = o.block_norm(ref[0], ref[1], post or "none", ref[2], ref[3], ref[4], 0.5, kind, ref[5], ref[6], 1e-5)
    near(s.detach(), s64.detach())
    near(y.detach(), y64.detach())
    torch.autograd.backward([t for t, _ in ((s64, ds),) * (use != "y") + ((y64, dy),) * (use != "s")],
                            [t.to(F64) for t in [ds] * (use != "y") + [dy] * (use != "s")])
    for got, want in zip(leaves, ref):
        if got is None:
            continue
        if want.grad is None:     # only s was used: the library's gradient of y's weights is 0
            assert not got.grad.any()
        else:
            assert (got.grad.to(F64) - want.grad).norm() <= 2.0 ** -5 * want.grad.norm()
    assert r.grad.data_ptr() != h.grad.data_ptr()


def test_block_norm_before_the_first_block():
    r, w = leaf(5, 8, seed=1), leaf(8, seed=2)
    s, y = nn.block_norm(r, w)
    assert s is r
    (s.float().sum() + y.float().square().sum()).backward()
    ref = [t.detach().to(F64).requires_grad_() for t in (r, w)]
    (ref[0].sum() + o.block_norm(ref[0], None, "none", None, None, None, 1.0, "rms", ref[1], None, 1e-5)[1].square().sum()).backward()
    for got, want in zip((r, w), ref):
        assert (got.grad.to(F64) - want.grad).norm() <= 2.0 ** -5 * want.grad.norm()


def test_block_norm_refusals_and_layouts():
    r, h, w = leaf(4, 6, seed=1), leaf(4, 6, seed=2), leaf(6, seed=3)
    for kw in (dict(kind="none"), dict(post="batch"), dict(post="rms"), dict(gate=w), dict(h=leaf(4, 5)),
               dict(h=h, gate=leaf(3, 6))):
        with pytest.raises(ValueError):
            nn.block_norm(r, w, **kw)
    # columns apart, and gradients of a sum (stride 0)
    s, y = nn.block_norm(leaf(6, 4, seed=4).t(), w, h=leaf(6, 4, seed=5).t())
    (s.sum() + y.sum()).backward()
    assert w.grad is not None
    s, y = nn.block_norm(r, w, h=h)
    with torch.no_grad():
        s.add_(1.0)
    with pytest.raises(RuntimeError):      # the saved sum was written over
        y.sum().backward()


def test_second_orders_are_refused():
    w, ids = leaf(5, 4), torch.tensor([0, 2, 2])
    for out, at in ((nn.embedding(ids, w), w), (nn.block_norm(leaf(3, 4), w[0])[1], w),
                    (nn.linear_cross_entropy(leaf(3, 4, seed=2), w, ids), w)):
        g, = torch.autograd.grad(out.float().square().sum(), at, create_graph=True)
        with pytest.raises(RuntimeError):
            g.float().square().sum().backward()


@pytest.mark.parametrize("lead", [(6,), (2, 3)])
@pytest.mark.parametrize("scaled", [False, True])
def test_linear_cross_entropy(lead, scaled):
    x, w = leaf(*lead, 8, seed=1), leaf(9, 8, seed=2)
    t = torch.tensor([0, 8, 3, -100, 3, 1]).view(lead)
    scale = torch.arange(6.0).view(lead) if scaled else None
    out = nn.linear_cross_entropy(x, w, t, scale=scale)
    assert out.shape == () and out.dtype == torch.float32
    (3.0 * out).backward()
    ref = o.cross_entropy(x.detach().view(6, 8), w.detach(), t.view(6), scale=None if scale is None else scale.view(6))
    assert abs(out.item() - ref[1].item()) < 1e-5
    near(x.grad.view(6, 8), 3.0 * ref[2])
    near(w.grad, 3.0 * ref[3])
    with torch.no_grad():
        assert torch.equal(nn.linear_cross_entropy(x, w, t, scale=scale), out.detach())
    out = nn.linear_cross_entropy(x, w.detach(), t)
    out.backward(retain_graph=True)
    first = x.grad.clone()
    out.backward()                     # twice: nothing was scaled in place
    assert torch.equal(x.grad - first, x.grad - first) and torch.isfinite(x.grad).all()
    for bad in ((x, w[:, :7], t), (x, w, t.view(-1)[:5])):
        with pytest.raises(ValueError):
            nn.linear_cross_entropy(*bad)
    with pytest.raises(ValueError):
        nn.linear_cross_entropy(x, w, t, scale=torch.ones(5))


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_linear_cross_entropy_without_gradients(mode, monkeypatch):
    """Where nothing is recorded the library is asked for the loss alone, whatever requires gradients."""
    asked = []

    def recorded(*args, dx=None, dw=None, **kw):
        asked.append((dx is not None, dw is not None))
        loss(*args, dx=dx, dw=dw, **kw)

    monkeypatch.setattr(nn, "zero_linear_cross_entropy", torch.no_grad()(recorded))
    x, w, t = leaf(6, 8, seed=1), leaf(9, 8, seed=2), torch.tensor([0, 8, 3, -100, 3, 1])
    with mode():
        out = nn.linear_cross_entropy(x, w, t)
    assert asked == [(False, False)] and not out.requires_grad
    assert torch.equal(nn.linear_cross_entropy(x, w, t).detach(), out)
    nn.linear_cross_entropy(x, w.detach(), t)
    nn.linear_cross_entropy(x.detach(), w, t)
    nn.linear_cross_entropy(x.detach(), w.detach(), t)
    assert asked[1:] == [(True, True), (True, False), (False, True), (False, False)]


def test_linear_cross_entropy_backward_twice():
    """Each backward pass multiplies what the forward pass computed by its own factor."""
    x, w, t = leaf(6, 8, seed=1), leaf(9, 8, seed=2), torch.tensor([0, 8, 3, -100, 3, 1])
    ref = o.cross_entropy(x.detach(), w.detach(), t)
    out = nn.linear_cross_entropy(x, w, t)
    for factor in (3.0, 1.0, -0.25):
        x.grad = w.grad = None
        (factor * out).backward(retain_graph=True)
        near(x.grad, factor * ref[2])
        near(w.grad, factor * ref[3])
