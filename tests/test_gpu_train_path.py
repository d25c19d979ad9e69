"""The training step as a user runs it: autograd over the library's linear maps, clipping and
AdamW together."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import train_oracle as o
import zero_partitioned_mixed_adam_gb300 as za
from zero_partitioned_mixed_adam_gb300.nn import linear
from zero_partitioned_mixed_adam_gb300.optim import TensorAdamW

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def leaf(*shape, sigma=1.0, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=gen) * sigma).bfloat16().requires_grad_()


def act64(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return torch.nn.functional.gelu(z, approximate="tanh")
    return torch.nn.functional.silu(z) if name == "silu" else z


@pytest.mark.parametrize("act", [None, "relu", "gelu", "silu"])
@pytest.mark.parametrize("lead", [(40,), (3, 50), (2, 1)])
def test_autograd_against_64_bits(act, lead):
    x, w, b = leaf(*lead, 96, seed=1), leaf(136, 96, sigma=0.1, seed=2), leaf(136, seed=3)
    r, dy = leaf(*lead, 136, seed=4), leaf(*lead, 136, seed=5).detach()
    y = linear(x, w, b, act, r)
    y.backward(dy)
    ref = [t.detach().double().requires_grad_() for t in (x, w, b, r)]
    z = act64(ref[0] @ ref[1].t() + ref[2], act) + ref[3]
    z.backward(dy.double())
    assert y.shape == z.shape
    # bf16 results of bf16 intermediates (pre, dz): a few roundings of 2^-9 each
    for got, want in zip((y, x.grad, w.grad, b.grad, r.grad), (z, *(t.grad for t in ref))):
        assert got.shape == want.shape
        assert (got.double() - want).norm() <= 2.0 ** -6 * want.norm()


def test_only_what_is_asked_for():
    x, w = leaf(20, 64, seed=1).detach(), leaf(32, 64, seed=2)
    linear(x, w, None, "gelu").sum().backward()
    assert x.grad is None and w.grad is not None
    x = leaf(64, 20, seed=1)
    y = linear(x.t(), w.detach())           # columns not contiguous: copied
    y.sum().backward()
    assert torch.equal(x.grad, w.detach().float().sum(0).bfloat16()[:, None].expand(64, 20)) or \
        (x.grad.float() - w.detach().float().sum(0)[:, None]).abs().max() <= 2.0 ** -7 * 10
    with pytest.raises(ValueError):
        linear(x, w)
    with pytest.raises(ValueError):
        linear(x.t(), w, act="tanh")
    with pytest.raises(ValueError):
        linear(x.t(), w, residual=x)


@pytest.mark.parametrize("eight", [False, True])
def test_optimizer_against_64_bits(eight):
    """Three clipped steps of TensorAdamW with fp32 moments follow AdamW in 64 bits; with 8-bit
    moments each weight is within a step's size of it."""
    params = [leaf(70, 33, sigma=0.1, seed=1).detach(), leaf(33, sigma=0.1, seed=2).detach()]
    opt = TensorAdamW(params, lr=1e-2, betas=(0.9, 0.95), weight_decay=0.1, max_norm=0.5, eight_bit=eight)
    w = [p.double().cpu().numpy() for p in params]
    m, v = [np.zeros_like(x) for x in w], [np.zeros_like(x) for x in w]
    for t in range(1, 4):
        for i, p in enumerate(params):
            p.grad = leaf(*p.shape, sigma=0.1, seed=10 * t + i).detach()
        opt.step()
        g = [p.grad.double().cpu().numpy() for p in params]
        norm = np.sqrt(sum((x ** 2).sum() for x in g))
        c = min(1.0, 0.5 / (norm + 1e-6))
        assert abs(opt.norm[0].item() - norm) <= 1e-5 * norm
        for i in range(2):
            m[i] = 0.9 * m[i] + 0.1 * c * g[i]
            v[i] = 0.95 * v[i] + 0.05 * (c * g[i]) ** 2
            w[i] = o.update(w[i], m[i], v[i], 1e-2, 0.1 if i == 0 else 0.0, 0.9, 0.95, 1e-8, t)
            # 8 bits: each moment off by at most a step, 1/8 of it, and the update, at most
            # about lr a step, by a quarter of itself and more where v is small
            tol = 1e-2 * t if eight else 1e-5 * np.abs(w[i]) + 1e-6
            assert (np.abs(opt.master[i].cpu().numpy() - w[i]) <= tol).all()
            assert torch.equal(params[i], opt.master[i].bfloat16())
    mm, vv = opt.moments()
    assert all(x.dtype == torch.float32 for x in mm + vv)
    n = sum(p.numel() for p in params)
    assert opt.state_bytes() == (6 * n + 8 * 11 if eight else 12 * n)
    opt.zero_grad()
    assert not any(p.grad.any() for p in params)


def test_optimizer_refusals():
    with pytest.raises(ValueError):
        TensorAdamW([torch.zeros(3)], lr=1e-3)
    with pytest.raises(ValueError):
        TensorAdamW([torch.zeros(3, device="cuda")], lr=1e-3)
    opt = TensorAdamW([leaf(8)], lr=1e-3)
    with pytest.raises(ValueError):
        opt.step()


@pytest.mark.parametrize("eight", [False, True])
def test_example_learns(eight):
    spec = importlib.util.spec_from_file_location("train_mlp", os.path.join(ROOT, "examples", "train_mlp.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses = mod.train(steps=60, eight_bit=eight)
    assert losses[-1] < 0.5 * losses[0]
    assert za.device_status() == za.ZERO_OK


@pytest.mark.parametrize("eight", [False, True])
def test_a_replaced_parameter_is_the_one_stepped(eight):
    """p.data = ... between two steps with the same gradient buffers: the new storage gets the
    weights, the old one is left alone."""
    params = [leaf(70, 33, seed=1).detach(), leaf(33, seed=2).detach()]
    grads = [leaf(70, 33, seed=3).detach(), leaf(33, seed=4).detach()]
    opt = TensorAdamW(params, lr=1e-2, eight_bit=eight, grads=grads)
    opt.step()
    old, before = params[0].data, params[0].clone()
    params[0].data = torch.zeros_like(old)
    opt.step()
    assert torch.equal(old, before)
    for p, w in zip(params, opt.master):
        assert torch.equal(p, w.bfloat16())


def test_moments_between_steps():
    """The values of 8-bit moments with the gradients set to None, and before the first step."""
    params = [leaf(70, 33, seed=1).detach(), leaf(33, seed=2).detach()]
    opt = TensorAdamW(params, lr=1e-2, eight_bit=True)
    assert not any(x.any() for xs in opt.moments() for x in xs)
    for p in params:
        p.grad = torch.ones_like(p)
    opt.step()
    for p in params:
        p.grad = None
    m, v = opt.moments()
    for x, want in ((m, 0.1), (v, 1e-3)):      # 3 bits after the first, rounded either way
        assert all(((t / want - 1.0).abs() <= 2.0 ** -3).all() for t in x)


def test_8bit_optimizer_step_by_step():
    """With 8-bit moments each step is AdamW in 64 bits on the moments' values before it, to
    binary32's roundings (16 operations of 2^-22, on the magnitudes that m is a sum of), as the
    weights take the new moments before they are encoded; and the new values are within one
    step of their codes of the exact ones: 1/8, or the least step of the block."""
    params = [leaf(70, 33, sigma=0.1, seed=1).detach(), leaf(33, sigma=0.1, seed=2).detach()]
    opt = TensorAdamW(params, lr=1e-2, betas=(0.9, 0.95), weight_decay=0.1, max_norm=0.5, eight_bit=True)
    for t in range(1, 6):
        for i, p in enumerate(params):
            p.grad = leaf(*p.shape, sigma=0.1, seed=10 * t + i).detach()
        before = [[x.double().cpu().numpy() for x in xs] for xs in (*opt.moments(), opt.master)]
        opt.step()
        c = float(opt.norm[1])
        assert 0.0 < c < 1.0
        after = [[x.double().cpu().numpy() for x in xs] for xs in (*opt.moments(), opt.master)]
        for i, p in enumerate(params):
            m, v, w = (x[i] for x in before)
            g = c * p.grad.double().cpu().numpy()
            size = 0.9 * np.abs(m) + 0.1 * np.abs(g)
            m, v = 0.9 * m + 0.1 * g, 0.95 * v + 0.05 * g * g
            decay = 0.1 if i == 0 else 0.0
            want = o.update(w, m, v, 1e-2, decay, 0.9, 0.95, 1e-8, t)
            most = np.abs(o.update(np.zeros_like(w), size, v, 1e-2, 0.0, 0.9, 0.95, 1e-8, t))
            got = after[2][i]
            assert (np.abs(got - want) <= 16 * 2.0 ** -22 * most + 2.0 ** -23 * (np.abs(w) + np.abs(want))).all()
            # a first step is about lr in size; an untouched weight would be that far off
            assert (np.abs(got - w) > 1e-4).mean() > 0.8
            for x, exact, least in ((after[0][i], m, 2.0 ** -17), (after[1][i], v, 2.0 ** -33)):
                x, exact = x.ravel(), exact.ravel()
                scale = np.repeat([np.abs(exact[b:b + o.BLOCK]).max() * 17 / 16 for b in range(0, len(exact), o.BLOCK)],
                                  o.BLOCK)[:len(exact)]
                step = np.maximum(2.0 ** -3 * np.abs(exact), least * scale)
                assert (np.abs(x - exact) <= step * (1 + 2.0 ** -16)).all()
