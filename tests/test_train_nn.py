"""nn.linear's autograd function on the host: the two library calls are replaced by products in
64 bits that take their arguments as the library does."""
import pytest
import torch

from zero_partitioned_mixed_adam_gb300 import nn, train_ops


def as_the_library(*matrices):
    for t in matrices:
        if t is not None and train_ops._matrix("matrix", t, *t.shape) < t.shape[1]:
            raise RuntimeError("a pitch below the width")


def forward(x, w, y, *, bias=None, act=0, residual=None, pre=None):
    as_the_library(x, w, y, residual, pre)
    assert act == 0 and pre is None
    z = x.double() @ w.double().t()
    if bias is not None:
        train_ops._vector("bias", bias, w.shape[0])
        z = z + bias.double()
    y.copy_(z if residual is None else z + residual.double())


def backward(dy, x, w, *, dx=None, dw=None, dbias=None, act=0, pre=None):
    as_the_library(dy, x, w, dx, dw)
    for out, value in ((dx, lambda: dy.double() @ w.double()),
                       (dw, lambda: dy.double().t() @ x.double()),
                       (dbias, lambda: dy.double().sum(0))):
        if out is not None:
            out.copy_(value())


@pytest.fixture(autouse=True)
def on_the_host(monkeypatch):
    monkeypatch.setattr(nn, "zero_linear_forward", torch.no_grad()(forward))
    monkeypatch.setattr(nn, "zero_linear_backward", torch.no_grad()(backward))


def leaf(*shape, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=gen).bfloat16().requires_grad_()


def test_second_order_gradients_are_refused():
    """A gradient penalty needs the backward pass's own gradient, which the library does not
    have: asking for it is an error, not a gradient without the penalty's part."""
    x, w = leaf(5, 8, seed=1), leaf(6, 8, seed=2)
    y = nn.linear(x, w)
    dx, = torch.autograd.grad(y.float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        (dx.float().square().sum() + y.float().sum()).backward()
    first = torch.autograd.grad(nn.linear(x, w).float().sum(), (x, w), create_graph=True)
    assert [g.shape for g in first] == [x.shape, w.shape]     # the first order is there as ever


def reference(x, w, b=None, r=None):
    x, w, b, r = (t if t is None else t.detach().double().requires_grad_() for t in (x, w, b, r))
    z = x @ w.t()
    z = z if b is None else z + b
    return (z if r is None else z + r), (x, w, b, r)


def near(got, want):
    assert got.shape == want.shape
    assert (got.double() - want).abs().max() <= 2.0 ** -7 * want.abs().max()


@pytest.mark.parametrize("out", [1, 6])
def test_expanded_gradients(out):
    """The gradient of a sum over rows has the row stride 0; that of a whole sum, both."""
    x, w, c = leaf(5, 8, seed=1), leaf(out, 8, seed=2), leaf(out, seed=3).detach()
    for loss in (lambda y: (y.sum(0) * c.to(y.dtype)).sum(), lambda y: y.sum()):
        x.grad = w.grad = None
        loss(nn.linear(x, w)).backward()
        z, (rx, rw, _, _) = reference(x, w)
        loss(z).backward()
        near(x.grad, rx.grad)
        near(w.grad, rw.grad)


@pytest.mark.parametrize("width", [1, 8])
def test_expanded_and_overlapping_inputs(width):
    w, b, r = leaf(6, width, seed=2), leaf(1, seed=3).expand(6), leaf(6, seed=4).expand(5, 6)
    rows = leaf(width + 4, seed=1)
    for x in (leaf(width, seed=1).expand(5, width), rows.unfold(0, width, 1)):
        y = nn.linear(x, w, b, residual=r)
        near(y, reference(x, w, b, r)[0])
    v = leaf(width, seed=1)
    nn.linear(v.expand(5, width), w).sum().backward()
    want, (rx, _, _, _) = reference(v.expand(5, width), w)
    want.sum().backward()
    near(v.grad, rx.grad.sum(0))
    row = leaf(width, seed=5)
    near(nn.linear(leaf(5, width), row.expand(6, width)), reference(leaf(5, width), row.expand(6, width))[0])


@pytest.mark.parametrize("lead", [(5,), (2, 3), ()])
def test_in_place_on_the_output(lead):
    """The output is a tensor of its own, which may be written in place like any other."""
    x, w = leaf(*lead, 8, seed=1), leaf(6, 8, seed=2)
    y = nn.linear(x, w)
    near(y.mul_(2.0).add_(1.0), 2 * reference(x, w)[0] + 1)
    y.sum().backward()
    z, (rx, rw, _, _) = reference(x, w)
    (2 * z).sum().backward()
    near(x.grad, rx.grad)
    near(w.grad, rw.grad)
