"""nn.linear on the GPU with the tensors that losses and broadcasts make."""
import pytest
import torch

from zero_partitioned_mixed_adam_gb300.nn import linear

pytestmark = pytest.mark.gpu


def leaf(*shape, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=gen).bfloat16().requires_grad_()


def near(got, want):
    """bf16 results of bf16 operands: up to two roundings of 2^-9 (a broadcast input's gradient
    is summed from rounded rows), fp32 sums' errors far less."""
    assert got.shape == want.shape
    assert (got.double() - want).abs().max() <= (2.0 ** -8 + 2.0 ** -16) * want.abs().max()


@pytest.mark.parametrize("out", [1, 72])
def test_expanded_tensors(out):
    """x and the residual broadcast over rows, the loss a sum over rows: strides of 0."""
    row, w, r, c = leaf(96, seed=1), leaf(out, 96, seed=2), leaf(out, seed=3), leaf(out, seed=4).detach()
    x = leaf(40, 96, seed=5)
    for a in (row.expand(40, 96), x):
        y = linear(a, w, residual=r.expand(40, out))
        z = a.detach().double() @ w.detach().double().t() + r.detach().double()
        near(y, z)
        for t in (row, w, r, x):
            t.grad = None
        (y.sum(0) * c).sum().backward()
        near(w.grad, c.double()[:, None] * a.detach().double().sum(0))
        near(r.grad, 40 * c.double())
        dx = (c.double() @ w.detach().double()).expand(40, 96)
        near(*((x.grad, dx) if a is x else (row.grad, dx.sum(0))))


def test_in_place_on_the_output():
    x, w = leaf(4, 10, 96, seed=1), leaf(72, 96, seed=2)
    z = x.detach().double() @ w.detach().double().t()
    y = linear(x, w).relu_()
    near(y, z.clamp(min=0))
    y.sum().backward()
    near(w.grad, ((z > 0).double().flatten(0, 1).t() @ x.detach().double().flatten(0, 1)))
