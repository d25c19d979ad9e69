"""What TensorAdamW hands to the library, on the host (its constructor wants CUDA tensors; the
list that it marshals only has their addresses)."""
import pytest
import torch

import zero_partitioned_mixed_adam_gb300 as za
from zero_partitioned_mixed_adam_gb300 import optim


def optimizer(eight=False, sizes=(300, 40), grads=None):
    opt = object.__new__(optim.TensorAdamW)
    opt.params = [torch.randn(n).bfloat16() for n in sizes]
    opt.master = [p.float() for p in opt.params]
    kind = torch.uint8 if eight else torch.float32
    opt.m, opt.v = ([torch.zeros(n, dtype=kind) for n in sizes] for _ in range(2))
    opt.m_scale, opt.v_scale = ([torch.zeros(-(-n // za.ZERO_MOMENT_BLOCK)) for n in sizes] if eight else None
                                for _ in range(2))
    opt.decay, opt.eight_bit, opt.grads, opt._list = [0.0] * len(sizes), eight, grads, None
    if grads is None:
        for p in opt.params:
            p.grad = torch.zeros_like(p)
    return opt


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("own_grads", [False, True])
def test_replaced_storage_is_noticed(eight, own_grads):
    grads = [torch.zeros(300), torch.zeros(40)] if own_grads else None
    opt = optimizer(eight, grads=grads)
    lst = opt._tensors()
    assert opt._tensors() is lst                     # nothing has moved
    fields = [("params", "param_bf16"), ("master", "master"), ("m", "m"), ("v", "v")]
    fields += [("m_scale", "m_scale"), ("v_scale", "v_scale")] if eight else []
    for column, field in fields:
        t = getattr(opt, column)[1]
        before, t.data = t.data, t.data.clone()      # the old storage lives on, as memory may not
        new = opt._tensors()
        assert getattr(new.arr[1], field) == t.data_ptr() != before.data_ptr(), column
        assert opt._tensors() is new
        setattr(opt, column, [x.clone() for x in getattr(opt, column)])
        if column == "params" and not own_grads:
            for p in opt.params:
                p.grad = torch.zeros_like(p)
        assert getattr(opt._tensors().arr[0], field) == getattr(opt, column)[0].data_ptr(), column
    g = opt.grads if own_grads else [p.grad for p in opt.params]
    g[0].data = g[0].data.clone()
    assert opt._tensors().arr[0].grad == g[0].data_ptr()
    if own_grads:
        opt.grads = grads + [torch.zeros(3)]
        with pytest.raises(ValueError):              # one gradient too many
            opt._tensors()


def test_moments_need_no_gradients(monkeypatch):
    """A checkpoint is taken between steps, where gradients are usually None."""
    opt, calls = optimizer(eight=True), []
    monkeypatch.setattr(optim, "zero_adamw_state_f32", lambda lst, m, v: calls.append((lst, m, v)))
    for p in opt.params:
        p.grad = None
    m, v = opt.moments()
    (lst, *outs), = calls
    assert outs[0] is m and outs[1] is v and lst.flags & za.ZERO_STATE_8BIT
    for i, p in enumerate(opt.params):
        assert m[i].shape == v[i].shape == p.shape and lst.arr[i].numel == p.numel()
        assert lst.arr[i].m == opt.m[i].data_ptr() and lst.arr[i].v_scale == opt.v_scale[i].data_ptr()
    with pytest.raises(ValueError):
        opt._tensors()                               # a step does need them


def test_a_grad_scale_of_another_type_is_refused():
    """The step reads 4 bytes of it as fp32, whatever they are."""
    opt = optimizer()
    for bad in (torch.tensor([0.5]).bfloat16(), torch.tensor([0.5], dtype=torch.float64), torch.tensor([1]),
                torch.zeros(0)):
        with pytest.raises(ValueError):
            za.zero_adamw_step(opt._tensors(), lr=1e-3, t=1, grad_scale=bad)
    none = za.adamw_tensors([], [], [], [])
    for good in (None, torch.tensor(0.5), torch.tensor([0.5]), torch.ones(2)[1:], 1 << 40):
        za.zero_adamw_step(none, lr=1e-3, t=1, grad_scale=good)     # nothing to step: no launch
