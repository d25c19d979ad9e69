"""The library's operators for PyTorch's autograd, over its forward and backward calls.

linear(x, weight, bias, act, residual) is act(x weight^T + bias) + residual in one launch;
embedding, block_norm and linear_cross_entropy are a model's two ends and what stands between
its blocks.  The backward passes are the library's; a gradient of one (a second order) is
refused.  Everything is bf16 on the GPU with fp32 sums.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (ZERO_ACT_GELU, ZERO_ACT_NONE, ZERO_ACT_RELU, ZERO_ACT_SILU, ZERO_NORM_LAYER,
               ZERO_NORM_NONE, ZERO_NORM_RMS, zero_block_norm_backward, zero_block_norm_forward,
               zero_embedding_backward, zero_embedding_forward, zero_linear_backward,
               zero_linear_cross_entropy, zero_linear_forward)

ACTS = {None: ZERO_ACT_NONE, "none": ZERO_ACT_NONE, "relu": ZERO_ACT_RELU, "gelu": ZERO_ACT_GELU,
        "silu": ZERO_ACT_SILU}
NORMS = {None: ZERO_NORM_NONE, "none": ZERO_NORM_NONE, "rms": ZERO_NORM_RMS, "layer": ZERO_NORM_LAYER}


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


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, ids, scale, padding):
        vocab, width = weight.shape
        y = torch.empty((*ids.shape, width), dtype=torch.bfloat16, device=weight.device)
        flat = ids.reshape(-1).contiguous()
        zero_embedding_forward(flat, _rows(weight, width), y.view(-1, width), scale=scale)
        ctx.save_for_backward(flat)
        ctx.shape, ctx.scale, ctx.padding = weight.shape, scale, padding
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        ids, = ctx.saved_tensors
        dy = _rows(grad, ctx.shape[1])
        dw = torch.empty(ctx.shape, dtype=torch.bfloat16, device=dy.device)
        zero_embedding_backward(dy, ids, dw, scale=ctx.scale, padding=ctx.padding)
        return dw, None, None, None


def embedding(ids, weight, scale: float = 1.0, padding_idx=None):
    """scale * weight[ids] for ids of any shape (int64 or int32) and weight [vocab, width], bf16.
    Rows whose id is padding_idx have no gradient.  Ids outside the table give NaN."""
    if weight.dim() != 2 or ids.dtype not in (torch.int64, torch.int32):
        raise ValueError(f"weight is a matrix and ids are int64 or int32, not {tuple(weight.shape)} and {ids.dtype}")
    return _Embedding.apply(weight, ids, float(scale), padding_idx)


class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, r, h, post_weight, post_bias, gate, weight, bias, post, kind, alpha, eps):
        width = r.shape[-1]
        flat = _rows(r, width)
        y = torch.empty(r.shape, dtype=torch.bfloat16, device=r.device)
        vectors = [None if t is None else t.contiguous() for t in (post_weight, post_bias, weight, bias)]
        if gate is not None:
            gate = gate.contiguous() if gate.dim() == 1 else _rows(gate, width)
        ctx.kinds = dict(post=post, kind=kind, alpha=alpha, eps=eps)
        if h is None:
            s, out, block = flat, None, None
        else:
            out = torch.empty(r.shape, dtype=torch.bfloat16, device=r.device)
            s, block = out.view(-1, width), _rows(h, width)
        zero_block_norm_forward(flat, y.view(-1, width), h=block, s=None if out is None else s, post_weight=vectors[0],
                                post_bias=vectors[1], gate=gate, weight=vectors[2], bias=vectors[3], **ctx.kinds)
        # (s as the output itself where it is one, so that writing it in place is noticed)
        ctx.save_for_backward(flat if out is None else out, block, gate, *vectors[:3])
        ctx.shape, ctx.has_bias, ctx.gate_shape = r.shape, bias is not None, None if gate is None else gate.shape
        ctx.set_materialize_grads(False)
        return y if out is None else (out, y)

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        s, block, gate, w1, b1, w = ctx.saved_tensors
        width = ctx.shape[-1]
        ds, dy = (None, grads[0]) if block is None else grads
        if ds is None and dy is None:
            return (None,) * 11
        need = ctx.needs_input_grad
        s = s.view(-1, width) if block is not None else s

        def rows(t):
            return None if t is None else _rows(t, width)

        def like(wanted, shape):
            return torch.empty(shape, dtype=torch.bfloat16, device=s.device) if wanted else None

        dr, dh = like(need[0], s.shape), like(need[1], s.shape)
        dw1, db1 = like(need[2], (width,)), like(need[3], (width,))
        dg = like(need[4], ctx.gate_shape)
        dw, db = like(need[5], (width,)), like(need[6] and ctx.has_bias, (width,))
        dy = rows(dy) if dy is not None else torch.zeros_like(s)
        zero_block_norm_backward(dy, s, ds=rows(ds), h=block, post_weight=w1, post_bias=b1, gate=gate, weight=w, dr=dr,
                                 dh=dh, dgate=dg, dpost_weight=dw1, dpost_bias=db1, dweight=dw, dbias=db, **ctx.kinds)

        def shaped(t):
            return None if t is None else t.view(ctx.shape)

        if dg is not None and dg.dim() == 2:
            dg = shaped(dg)
        return shaped(dr), shaped(dh), dw1, db1, dg, dw, db, None, None, None, None


def block_norm(r, weight=None, bias=None, *, h=None, kind="rms", post=None, post_weight=None, post_bias=None,
               gate=None, alpha: float = 1.0, eps: float = 1e-5):
    """(s, y) with s = r + alpha * gate * P(h) and y = N(s): the residual stream r takes the output h
    of a block, and the next block gets y, all in one launch.  Without h (before the first block)
    s is r.

    r, h [..., width], bf16; N: kind "rms" or "layer" with weight and bias [width]; P: the norm
    after the block, post None, "rms" or "layer" with post_weight and post_bias; gate: [width] or
    of h's shape."""
    if kind not in ("rms", "layer") or post not in NORMS:
        raise ValueError(f'kind: "rms" or "layer", post: one of {list(NORMS)}; not {kind!r} and {post!r}')
    if h is None and (gate is not None or NORMS[post] != ZERO_NORM_NONE):
        raise ValueError("a gate and a norm after the block need the block's output h")
    for name, t in (("h", h), ("gate", gate if gate is not None and gate.dim() != 1 else None)):
        if t is not None and t.shape != r.shape:
            raise ValueError(f"{name}: expected {tuple(r.shape)}, got {tuple(t.shape)}")
    out = _BlockNorm.apply(r, h, post_weight, post_bias, gate, weight, bias, NORMS[post], NORMS[kind], float(alpha),
                           float(eps))
    return (r, out) if h is None else out


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, targets, ignore_index, scale, recorded):
        width = weight.shape[1]
        rows, w = _rows(x, width), _rows(weight, width)
        total = torch.empty(1, dtype=torch.float32, device=x.device)
        # (needs_input_grad says what requires gradients, whether or not anything is recorded)
        need_x, need_w = (recorded and need for need in ctx.needs_input_grad[:2])
        dx = torch.empty(rows.shape, dtype=rows.dtype, device=x.device) if need_x else None
        dw = torch.empty(w.shape, dtype=w.dtype, device=x.device) if need_w else None
        zero_linear_cross_entropy(rows, w, targets.reshape(-1).contiguous(), None, total, dx=dx, dw=dw,
                                  ignore_index=ignore_index,
                                  scale=None if scale is None else scale.reshape(-1).contiguous())
        ctx.save_for_backward(dx, dw)
        ctx.shape = x.shape
        return total.view(())

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        dx, dw = ctx.saved_tensors
        return (None if dx is None else (dx * grad).view(ctx.shape), None if dw is None else dw * grad, None, None,
                None, None)


def linear_cross_entropy(x, weight, targets, ignore_index: int = -100, scale=None):
    """The softmax cross entropy of x weight^T against targets, one number (fp32): the mean over
    rows whose target is not ignore_index, or with scale (fp32, of targets' shape) the sum of
    scale times each row's.  x [..., width], weight [vocab, width], bf16; targets of x's leading
    shape.  The logits are not kept: x's and weight's gradients are computed in the forward pass,
    where they are wanted (not under torch.no_grad), and only multiplied by the loss's own in the
    backward pass, which rounds them to bf16 once more unless that is a power of two."""
    if weight.dim() != 2 or x.shape[-1] != weight.shape[1] or targets.shape != x.shape[:-1]:
        raise ValueError(f"x {tuple(x.shape)}, weight {tuple(weight.shape)} and targets {tuple(targets.shape)} "
                         "do not match")
    if scale is not None and (scale.shape != targets.shape or scale.requires_grad):
        raise ValueError("scale is of targets' shape, and has no gradient")
    # asked here: within an autograd function nothing is ever recorded
    return _LinearCrossEntropy.apply(x, weight, targets, ignore_index, scale, torch.is_grad_enabled())
