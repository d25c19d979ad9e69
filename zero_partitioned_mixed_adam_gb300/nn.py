"""Linear maps for PyTorch's autograd, over zero_linear_forward and zero_linear_backward.

linear(x, weight, bias, act, residual) is act(x weight^T + bias) + residual in one launch, and
its backward pass the library's; a gradient of that (a second order) is refused.
Everything is bf16 on the GPU with fp32 sums.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (ZERO_ACT_GELU, ZERO_ACT_NONE, ZERO_ACT_RELU, ZERO_ACT_SILU, zero_linear_backward,
               zero_linear_forward)

ACTS = {None: ZERO_ACT_NONE, "none": ZERO_ACT_NONE, "relu": ZERO_ACT_RELU, "gelu": ZERO_ACT_GELU,
        "silu": ZERO_ACT_SILU}


def _rows(x, width):
    """x as a matrix with contiguous columns and rows that do not overlap (a copy only where
    it has to be: of columns apart, and of expanded tensors, whose strides are 0)."""
    x = x.reshape(-1, width)
    rows, pitch, step = x.shape[0], *x.stride()
    return x if (width == 1 or step == 1) and (rows <= 1 or pitch >= width) else x.contiguous()


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, act, residual):
        out, width = weight.shape
        rows = _rows(x, width)
        w = _rows(weight, width)
        # of x's shape from the start: a view made here could not be written in place
        y = torch.empty((*x.shape[:-1], out), dtype=torch.bfloat16, device=x.device)
        flat = y.view(-1, out)
        keep = act != ZERO_ACT_NONE and any(ctx.needs_input_grad[:3])
        pre = torch.empty_like(flat) if keep else None
        zero_linear_forward(rows, w, flat, act=act, pre=pre,
                            bias=None if bias is None else bias.contiguous(),
                            residual=None if residual is None else _rows(residual, out))
        ctx.save_for_backward(rows, w, pre)
        ctx.act, ctx.shape, ctx.has_bias = act, x.shape, bias is not None
        return y

    @staticmethod
    @once_differentiable  # the gradients of dx, dw and dbias are not the library's: no second order
    def backward(ctx, grad):
        rows, w, pre = ctx.saved_tensors
        need_x, need_w, need_b, _, need_r = ctx.needs_input_grad
        dy = _rows(grad, w.shape[0])
        dx = torch.empty(rows.shape, dtype=rows.dtype, device=rows.device) if need_x else None
        dw = torch.empty(w.shape, dtype=w.dtype, device=w.device) if need_w else None
        db = torch.empty(w.shape[0], dtype=w.dtype, device=w.device) \
            if need_b and ctx.has_bias else None
        if need_x or need_w or db is not None:
            zero_linear_backward(dy, rows, w, dx=dx, dw=dw, dbias=db, act=ctx.act, pre=pre)
        return (dx.view(ctx.shape) if need_x else None, dw, db, None, grad if need_r else None)


def linear(x, weight, bias=None, act=None, residual=None):
    """act(x weight^T + bias) + residual for x [..., in], weight [out, in], bias [out] and
    residual [..., out], all bf16; act: None, "relu", "gelu" (tanh form) or "silu"."""
    if act not in ACTS:
        raise ValueError(f"act: one of {list(ACTS)}, not {act!r}")
    if weight.dim() != 2 or x.shape[-1] != weight.shape[1]:
        raise ValueError(f"x {tuple(x.shape)} and weight {tuple(weight.shape)} do not match")
    if residual is not None and residual.shape != (*x.shape[:-1], weight.shape[0]):
        raise ValueError(f"residual: expected {(*x.shape[:-1], weight.shape[0])}, "
                         f"got {tuple(residual.shape)}")
    return _Linear.apply(x, weight, bias, ACTS[act], residual)
