"""A language model's training step with the library's operators from end to end: embedding, block
norms, linear maps, cross entropy, norm and AdamW together."""
import importlib.util
import os

import pytest
import torch

import model_oracle as o
import zero_partitioned_mixed_adam_gb300 as za
from zero_partitioned_mixed_adam_gb300 import nn

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F64 = torch.float64


@pytest.fixture(scope="module")
def lm():
    spec = importlib.util.spec_from_file_location("train_lm", os.path.join(ROOT, "examples", "train_lm.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def batch(vocab, tokens, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    ids = torch.randint(0, vocab, (tokens,), device="cuda", generator=gen)
    t = torch.randint(0, vocab, (tokens,), device="cuda", generator=gen)
    return ids, torch.where(torch.rand(tokens, device="cuda", generator=gen) < 0.2, -100, t)


def loss64(net, ids, targets, alpha):
    """The same model in 64 bits, with none of the library."""
    table = net["table"]
    s = table[ids] * table.shape[1] ** 0.5
    norms = [p["norm"] for p in net["blocks"]] + [net["norm"]]
    y = o.standardized(s, "rms", 1e-5)[0] * norms[0]
    for p, norm in zip(net["blocks"], norms[1:]):
        h = torch.nn.functional.gelu(y @ p["w1"].t() + p["b1"], approximate="tanh") @ p["w2"].t()
        s, y = o.block_norm(s, h, "rms", p["after"], None, p["gate"], alpha, "rms", norm, None, 1e-5)
    z = y @ table.t()
    keep = targets != -100
    return (torch.logsumexp(z, 1) - z.gather(1, targets.clamp(min=0)[:, None])[:, 0])[keep].mean()


@pytest.mark.parametrize("vocab,width,hidden,tokens", [(515, 256, 512, 300), (101, 75, 130, 64)])
def test_a_models_gradients(lm, vocab, width, hidden, tokens):
    net = lm.parameters(vocab, width, hidden, 2, torch.Generator("cuda").manual_seed(1))
    ids, targets = batch(vocab, tokens, 2)
    loss = lm.loss_of(net, ids, targets, 0.7)
    loss.backward()
    leaf = lambda t: t.detach().to(F64).requires_grad_()  # noqa: E731
    net64 = {"table": leaf(net["table"]), "norm": leaf(net["norm"]),
             "blocks": [{k: leaf(v) for k, v in p.items()} for p in net["blocks"]]}
    want = loss64(net64, ids, targets, 0.7)
    want.backward()
    # a dozen bf16 roundings of 2^-9 between a leaf and the loss, each on its own sum
    assert abs(loss.item() - want.item()) <= 2.0 ** -6
    for got, ref in zip(lm.tensors(net), lm.tensors(net64)):
        assert (got.grad.to(F64) - ref.grad).norm() <= 2.0 ** -4 * ref.grad.norm()
    assert za.device_status() == za.ZERO_OK


@pytest.mark.parametrize("eight", [False, True])
def test_example_runs(lm, eight):
    losses = lm.train(steps=12, eight_bit=eight)
    assert len(losses) == 3 and all(0.0 < x < 20.0 for x in losses)


def test_a_step_with_a_shared_table(lm):
    """The library's calls as a loop without autograd makes them: the loss writes the table's fp32
    gradient, the embedding's is added to it, and AdamW takes it, all on one side stream."""
    m, d, v = 200, 136, 700
    gen = torch.Generator("cuda").manual_seed(3)
    table = torch.randn(v, d, device="cuda", generator=gen) * d ** -0.5
    ids, targets = batch(v, m, 4)
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    param = table.bfloat16()
    e, y, dy, de = (torch.empty(m, d, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    grad, dw = torch.full((v, d), 7.0, device="cuda"), torch.full((d,), 7.0, device="cuda")
    total, norm = torch.empty(1, device="cuda"), torch.empty(2, device="cuda")
    ws = za.grad_norm_workspace()
    moments = [torch.zeros(v, d, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        za.zero_embedding_forward(ids, param, e, scale=d ** 0.5)
        za.zero_block_norm_forward(e, y, weight=w)
        za.zero_linear_cross_entropy(y, param, targets, None, total, dx=dy, dw=grad)
        za.zero_block_norm_backward(dy, e, weight=w, dr=de, dweight=dw)
        za.zero_embedding_backward(de, ids, grad, scale=d ** 0.5, accumulate=True)
        tensors = za.adamw_tensors([grad], [table], [moments[0]], [moments[1]], params=[param])
        before = param.clone()
        za.zero_grad_norm(tensors, norm, max_norm=1.0, workspace=ws)
        za.zero_adamw_step(tensors, lr=1e-2, t=1, grad_scale=norm[1:])
    torch.cuda.current_stream().wait_stream(side)
    t64 = before.to(F64).requires_grad_()
    w64 = w.to(F64).requires_grad_()
    y64 = o.standardized(t64[ids] * d ** 0.5, "rms", 1e-5)[0] * w64
    z = y64 @ t64.t()
    keep = targets != -100
    want = (torch.logsumexp(z, 1) - z.gather(1, targets.clamp(min=0)[:, None])[:, 0])[keep].mean()
    want.backward()
    assert abs(total.item() - want.item()) <= 2.0 ** -6
    assert (grad.to(F64) - t64.grad).norm() <= 2.0 ** -5 * t64.grad.norm()
    assert (dw.to(F64) - w64.grad).norm() <= 2.0 ** -5 * w64.grad.norm()
    assert abs(norm[0].item() - grad.to(F64).norm().item()) <= 1e-5 * norm[0].item()
    # a first step of AdamW is lr in size wherever there is a gradient
    moved = (table - before.float()).abs()
    assert (moved[grad != 0] <= 1.01e-2 + 2.0 ** -8 * before.float().abs().max()).all() and moved[grad != 0].mean() > 5e-3


def test_a_captured_step(lm):
    """Forward and backward of the whole model captured (after a warm-up on the capture's stream, no
    other graph of these leaves alive) and replayed on another batch: the eager bits."""
    net = lm.parameters(300, 128, 256, 1, torch.Generator("cuda").manual_seed(5))
    ids, targets = batch(300, 128, 6)
    flat = lm.tensors(net)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(lm.loss_of(net, ids, targets, 1.0), flat)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = lm.loss_of(net, ids, targets, 1.0)
        grads = torch.autograd.grad(loss, flat)
    new = batch(300, 128, 7)
    ids.copy_(new[0]), targets.copy_(new[1])
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (loss.detach(), *grads)]
    del loss, grads
    loss = lm.loss_of(net, ids, targets, 1.0)
    want = torch.autograd.grad(loss, flat)
    assert torch.equal(got[0], loss.detach()) and all(torch.equal(a, b) for a, b in zip(got[1:], want))


def test_two_graphs_do_not_share_a_workspace():
    """Calls captured into two graphs, replayed on two streams at once."""
    d, v, m = 256, 1031, 200
    gen = torch.Generator("cuda").manual_seed(8)
    w = (torch.randn(v, d, device="cuda", generator=gen) * 0.1).bfloat16()
    graphs, outs, eager, inputs = [], [], [], []
    for k in range(2):
        x = torch.randn(m, d, device="cuda", generator=gen).bfloat16()
        t = torch.randint(0, v, (m,), device="cuda", generator=gen)
        inputs.append((x, t))      # a graph does not keep them alive
        out = [torch.empty(1, device="cuda"), torch.empty_like(x), torch.empty_like(w), torch.empty(d, device="cuda")]

        def step(out=out, x=x, t=t):
            za.zero_linear_cross_entropy(x, w, t, None, out[0], dx=out[1], dw=out[2])
            za.zero_block_norm_backward(out[1], x, dweight=out[3])

        step()
        eager.append([a.clone() for a in out])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        graphs.append(graph)
        outs.append(out)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out, want in zip(outs, eager):
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_autograd_on_the_gpu():
    """nn's functions once each against 64 bits, with expanded and transposed tensors."""
    gen = torch.Generator("cuda").manual_seed(9)
    leaf = lambda *s: torch.randn(*s, device="cuda", generator=gen).bfloat16().requires_grad_()  # noqa: E731
    w, x = leaf(50, 24), leaf(24, 30)
    t = torch.randint(0, 50, (30,), device="cuda", generator=gen)
    loss = nn.linear_cross_entropy(x.t(), w, t)
    (2.0 * loss).backward()
    ref = o.cross_entropy(x.detach().t(), w.detach(), t)
    assert abs(loss.item() - ref[1].item()) <= 1e-4
    assert (x.grad.t().to(F64) - 2.0 * ref[2]).norm() <= 2.0 ** -6 * 2.0 * ref[2].norm()
    assert (w.grad.to(F64) - 2.0 * ref[3]).norm() <= 2.0 ** -6 * 2.0 * ref[3].norm()
    w.grad = None
    nn.embedding(t.view(5, 6), w).sum(0).sum().backward()          # a gradient of stride 0
    count = torch.bincount(t, minlength=50).to(F64)[:, None].expand(50, 24)
    assert torch.equal(w.grad.to(F64), count)
