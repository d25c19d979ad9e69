"""Binding of the training-step operators around the ZeRO step: a unit's linear maps forward
and backward, the global gradient norm, and AdamW over a list of tensors.

Like the rest of the binding it marshals arguments only; everything here is reached through
the package itself (zero_linear_forward, zero_grad_norm, zero_adamw_step, ...).
"""
from __future__ import annotations

import ctypes

import torch

from . import (ZERO_ACT_NONE, ZERO_GRAD_ACCUMULATE, ZERO_GRAD_F32, ZERO_LINEAR_ALIGNED,
               ZERO_LINEAR_BACKWARD, ZERO_LINEAR_PLAIN, ZERO_MOMENT_BLOCK, ZERO_OK, ZERO_STATE_8BIT,
               ZeroError, _addr, _lib, _ptrs, _stream_handle)


class ZeroLinear(ctypes.Structure):
    """zero_linear_t: sizes and row pitches of one linear map."""

    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "in_", "out", "ldx", "ldw", "ldy", "ldr",
                                              "ldp", "ldpi", "lddx", "lddw")]


class ZeroAdamwTensor(ctypes.Structure):
    """zero_adamw_tensor_t: one tensor of an AdamW list."""

    _fields_ = [("numel", ctypes.c_int64)] + [
        (n, ctypes.c_void_p) for n in ("grad", "master", "param_bf16", "m", "v", "m_scale",
                                       "v_scale")] + [("weight_decay", ctypes.c_double)]


def _declare(lib) -> None:
    vp, i32, i64, dbl = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double
    lin = ctypes.POINTER(ZeroLinear)
    lib.zero_linear_workspace.argtypes = [lin, i32]
    lib.zero_linear_workspace.restype = i64
    lib.zero_linear_forward.argtypes = [lin, vp, vp, vp, i32, vp, vp, vp, vp, i64, vp]
    lib.zero_linear_forward.restype = ctypes.c_int
    lib.zero_linear_backward.argtypes = [lin, vp, vp, vp, i32, vp, i32, vp, vp, vp, vp, i32, vp,
                                         i64, vp]
    lib.zero_linear_backward.restype = ctypes.c_int
    lib.zero_grad_norm_workspace.argtypes = []
    lib.zero_grad_norm_workspace.restype = i64
    lib.zero_grad_norm.argtypes = [i32, vp, vp, i32, dbl, vp, vp, i64, vp]
    lib.zero_grad_norm.restype = ctypes.c_int
    lib.zero_adamw_step.argtypes = [i32, vp, i32, dbl, dbl, dbl, dbl, i64, vp, ctypes.c_uint32, vp]
    lib.zero_adamw_step.restype = ctypes.c_int
    lib.zero_adamw_state_f32.argtypes = [i32, vp, vp, vp, vp]
    lib.zero_adamw_state_f32.restype = ctypes.c_int


_declare(_lib)

_BF16 = (torch.bfloat16,)
_GRADS = (torch.bfloat16, torch.float32)


# -------------------------------------------------------------------- linear maps

def _matrix(name, t, rows, cols, dtypes=_BF16):
    """A 2-D tensor's row pitch; its shape, strides and type checked."""
    if t.shape != (rows, cols):
        raise ValueError(f"{name}: expected {rows} x {cols}, got {tuple(t.shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: expected one of {dtypes}, got {t.dtype}")
    pitch, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name}: its columns are not contiguous (stride {step})")
    return pitch if rows > 1 else max(cols, pitch)


def _vector(name, t, n, dtypes=_BF16):
    if t.shape != (n,) or t.dtype not in dtypes or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name}: expected {n} contiguous elements of one of {dtypes}")


def _linear_workspace(shape, flags, bases, pitches, workspace, device, stream):
    """The caller's workspace, or one from PyTorch's allocator; and its bytes.  The allocator
    hands memory out, and takes it back, in the order of the stream that is current when it
    is asked, so it is asked on `stream`.  bases, pitches: those of the matrices (and the
    bias) that the products read, or-ed together."""
    if workspace is not None:
        return workspace, workspace.numel() * workspace.element_size()
    if bases % 16 == 0 and pitches % 8 == 0:
        flags |= ZERO_LINEAR_ALIGNED
    need = _lib.zero_linear_workspace(ctypes.byref(shape), flags)
    if need < 0:
        raise ZeroError(need, "zero_linear_workspace")
    if need == 0:
        return None, 0
    if stream is None:
        return torch.empty(need, dtype=torch.uint8, device=device), need
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device)
    with torch.cuda.stream(stream):
        return torch.empty(need, dtype=torch.uint8, device=device), need


def zero_linear_workspace(rows: int, width_in: int, width_out: int, backward: bool = False,
                          aligned: bool = False) -> int:
    """Bytes of workspace that suffice for a linear map of these sizes; aligned: of matrices
    (and a bias) that all start on 16-byte boundaries and have pitches that are multiples of 8."""
    flags = (ZERO_LINEAR_BACKWARD if backward else 0) | (ZERO_LINEAR_ALIGNED if aligned else 0)
    rc = _lib.zero_linear_workspace(ctypes.byref(ZeroLinear(rows, width_in, width_out)), flags)
    if rc < 0:
        raise ZeroError(rc, "zero_linear_workspace")
    return rc


def zero_linear_forward(x, w, y, *, bias=None, act: int = ZERO_ACT_NONE, residual=None, pre=None,
                        workspace=None, stream=None) -> None:
    """y = act(x w^T + bias) + residual, and pre = x w^T + bias where it is wanted.

    x [rows, in], w [out, in], y / residual / pre [rows, out]: bf16 tensors with
    contiguous columns and any row pitch (views of a unit's flat buffer among them);
    bias [out].  residual may be y itself.  Without a workspace tensor
    (zero_linear_workspace bytes) one is taken from PyTorch's allocator.
    """
    if x.dim() != 2 or y.dim() != 2:
        raise ValueError("x and y are matrices")
    (rows, out), k = y.shape, x.shape[1]
    s = ZeroLinear(rows, k, out, _matrix("x", x, rows, k), _matrix("w", w, out, k),
                   _matrix("y", y, rows, out))
    if bias is not None:
        _vector("bias", bias, out)
    if residual is not None:
        s.ldr = _matrix("residual", residual, rows, out)
    if pre is not None:
        s.ldp = _matrix("pre", pre, rows, out)
    px, pw, pb = x.data_ptr(), w.data_ptr(), _addr(bias)
    workspace, nbytes = _linear_workspace(s, 0, px | pw | (pb or 0), s.ldx | s.ldw, workspace,
                                          y.device, stream)
    rc = _lib.zero_linear_forward(ctypes.byref(s), px, pw, pb, act,
                                  _addr(residual), _addr(pre), _addr(y), _addr(workspace), nbytes,
                                  _stream_handle(stream))
    if rc != ZERO_OK:
        raise ZeroError(rc, "zero_linear_forward")


def zero_linear_backward(dy, x, w, *, dx=None, dw=None, dbias=None, act: int = ZERO_ACT_NONE,
                         pre=None, act_in: int = ZERO_ACT_NONE, pre_in=None,
                         accumulate: bool = False, workspace=None, stream=None) -> None:
    """Gradients of y = act(x w^T + bias): with dz = dy * act'(pre),
    dx = (dz w) * act_in'(pre_in), dw (+)= dz^T x, dbias (+)= dz summed over rows.

    Each of dx, dw and dbias that is given is written (dw and dbias added to with
    accumulate=True); dw and dbias are bf16 or fp32, both alike.  x may be None
    without dw, and w without dx.
    """
    if dy.dim() != 2:
        raise ValueError("dy is a matrix")
    if (dw is not None and x is None) or (dx is not None and w is None):
        raise ValueError("dw needs x, and dx needs w")
    rows, out = dy.shape
    k = next((t.shape[-1] for t in (x, w, dx) if t is not None), 1)
    s = ZeroLinear(rows, k, out)
    s.ldy = _matrix("dy", dy, rows, out)
    if x is not None:
        s.ldx = _matrix("x", x, rows, k)
    if w is not None:
        s.ldw = _matrix("w", w, out, k)
    if dx is not None:
        s.lddx = _matrix("dx", dx, rows, k)
    if dw is not None:
        s.lddw = _matrix("dw", dw, out, k, _GRADS)
    if dbias is not None:
        _vector("dbias", dbias, out, _GRADS)
        if dw is not None and dw.dtype != dbias.dtype:
            raise ValueError("dw and dbias have different types")
    if act != ZERO_ACT_NONE and pre is not None:
        s.ldp = _matrix("pre", pre, rows, out)
    if act_in != ZERO_ACT_NONE and pre_in is not None:
        s.ldpi = _matrix("pre_in", pre_in, rows, k)
    g = dw if dw is not None else dbias
    flags = ZERO_GRAD_F32 if g is not None and g.dtype == torch.float32 else 0
    if accumulate:
        flags |= ZERO_GRAD_ACCUMULATE
    workspace, nbytes = _linear_workspace(
        s, ZERO_LINEAR_BACKWARD | (ZERO_LINEAR_PLAIN if act == ZERO_ACT_NONE else 0),
        _addr(dy) | _addr(x) | _addr(w), s.ldy | s.ldx | s.ldw, workspace, dy.device, stream)
    rc = _lib.zero_linear_backward(ctypes.byref(s), _addr(dy), _addr(x), _addr(w), act, _addr(pre),
                                   act_in, _addr(pre_in), _addr(dx), _addr(dw), _addr(dbias),
                                   flags, _addr(workspace), nbytes, _stream_handle(stream))
    if rc != ZERO_OK:
        raise ZeroError(rc, "zero_linear_backward")


# ------------------------------------------------------------------ lists of tensors

class GradList:
    """A list of gradients, its addresses and sizes marshalled once (see grad_list)."""

    __slots__ = ("buffers", "ptrs", "numels", "flags")

    def __init__(self, grads):
        self.buffers = tuple(grads)
        kinds = {g.dtype for g in self.buffers}
        if len(kinds) > 1 or not kinds <= set(_GRADS):
            raise ValueError("the gradients are bf16 or fp32, all alike")
        if not all(g.is_contiguous() for g in self.buffers):
            raise ValueError("the gradients are contiguous")
        n = len(self.buffers)
        self.ptrs = (ctypes.c_void_p * max(n, 1))(*[_addr(g) for g in self.buffers])
        self.numels = (ctypes.c_int64 * max(n, 1))(*[g.numel() for g in self.buffers])
        self.flags = ZERO_GRAD_F32 if kinds == {torch.float32} else 0

    def __len__(self) -> int:
        return len(self.buffers)


def grad_list(grads) -> GradList:
    """A reusable list of gradients (bf16 or fp32 CUDA tensors) for zero_grad_norm.  Like a
    PointerArray it keeps the tensors alive and records their addresses as they are now."""
    return GradList(grads)


def grad_norm_workspace(device="cuda"):
    """A zeroed workspace for zero_grad_norm; each call leaves it ready for the next."""
    return torch.zeros(_lib.zero_grad_norm_workspace(), dtype=torch.uint8, device=device)


def zero_grad_norm(grads, out, *, max_norm: float, workspace, stream=None) -> None:
    """out[0] = the global 2-norm of the gradients, out[1] = min(1, max_norm / (norm + 1e-6)).

    grads: a GradList or an AdamwTensors; out: two fp32 on the device (out[1:] is
    zero_adamw_step's grad_scale); workspace: grad_norm_workspace()'s, one per stream."""
    if isinstance(grads, AdamwTensors):
        grads = grads.grads
    _vector("out", out, 2, (torch.float32,))
    rc = _lib.zero_grad_norm(len(grads), grads.ptrs, grads.numels, grads.flags, max_norm,
                             _addr(out), _addr(workspace),
                             workspace.numel() * workspace.element_size(), _stream_handle(stream))
    if rc != ZERO_OK:
        raise ZeroError(rc, "zero_grad_norm")


class AdamwTensors:
    """A list of tensors for zero_adamw_step, marshalled once (see adamw_tensors)."""

    __slots__ = ("grads", "buffers", "arr", "flags")

    def __init__(self, grads, masters, m, v, params=None, m_scale=None, v_scale=None,
                 weight_decay=0.0):
        self.grads = grads if isinstance(grads, GradList) else GradList(grads)
        n = len(self.grads)
        eight = m_scale is not None or v_scale is not None
        if eight and (m_scale is None or v_scale is None):
            raise ValueError("8-bit moments have both m_scale and v_scale")
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) \
            else [weight_decay] * n
        columns = [list(c) if c is not None else [None] * n
                   for c in (masters, params, m, v, m_scale, v_scale)]
        if any(len(c) != n for c in columns + [decay]):
            raise ValueError(f"expected {n} of each tensor")
        state = torch.uint8 if eight else torch.float32
        kinds = (torch.float32, torch.bfloat16, state, state, torch.float32, torch.float32)
        names = ("master", "param", "m", "v", "m_scale", "v_scale")
        for i, g in enumerate(self.grads.buffers):
            for name, kind, column in zip(names, kinds, columns):
                t = column[i]
                if t is None and (name == "param" or (name.endswith("scale") and not eight)):
                    continue
                want = g.numel()
                if name.endswith("scale"):
                    want = -(-want // ZERO_MOMENT_BLOCK)
                if t is None or t.dtype != kind or t.numel() != want or not t.is_contiguous():
                    raise ValueError(f"{name}[{i}]: expected {want} contiguous {kind} elements")
        self.buffers = columns
        self.flags = self.grads.flags | (ZERO_STATE_8BIT if eight else 0)
        self.arr = (ZeroAdamwTensor * max(n, 1))()
        for i, g in enumerate(self.grads.buffers):
            self.arr[i] = ZeroAdamwTensor(g.numel(), _addr(g), *[_addr(c[i]) for c in columns],
                                          decay[i])

    def __len__(self) -> int:
        return len(self.grads)


def adamw_tensors(grads, masters, m, v, *, params=None, m_scale=None, v_scale=None,
                  weight_decay=0.0) -> AdamwTensors:
    """A reusable list of tensors for zero_adamw_step: per tensor its gradient (bf16 or
    fp32), fp32 master weights, moments (fp32; or uint8 codes with fp32 m_scale and
    v_scale of ceil(numel / ZERO_MOMENT_BLOCK) elements, all zero to begin with), and
    optionally the bf16 parameter that is written.  weight_decay: one, or one each."""
    return AdamwTensors(grads, masters, m, v, params, m_scale, v_scale, weight_decay)


def zero_adamw_step(tensors: AdamwTensors, *, lr: float, beta1: float = 0.9, beta2: float = 0.999,
                    eps: float = 1e-8, t: int, grad_scale=None, seed: int = 0,
                    stream=None) -> None:
    """One AdamW step over a list of tensors (see zero_adamw_step in include/zeroadam.h).

    grad_scale: one fp32 on the device that multiplies every gradient, or None;
    seed: of the stochastic rounding of 8-bit moments, a new one every step."""
    if hasattr(grad_scale, "dtype") and (grad_scale.dtype != torch.float32 or grad_scale.numel() < 1):
        raise ValueError(f"grad_scale: expected one fp32, got {tuple(grad_scale.shape)} {grad_scale.dtype}")
    rc = _lib.zero_adamw_step(len(tensors), tensors.arr, tensors.flags, lr, beta1, beta2, eps, t,
                              _addr(grad_scale), seed & 0xFFFFFFFF, _stream_handle(stream))
    if rc != ZERO_OK:
        raise ZeroError(rc, "zero_adamw_step")


def zero_adamw_state_f32(tensors: AdamwTensors, m_out=None, v_out=None, stream=None) -> None:
    """The values of 8-bit moments as fp32, into one tensor each (as a checkpoint holds them)."""
    if not tensors.flags & ZERO_STATE_8BIT:
        raise ValueError("the moments of this list are fp32 already")
    arrays = []
    for name, out in (("m_out", m_out), ("v_out", v_out)):
        if out is None:
            arrays.append(None)
            continue
        if not hasattr(out, "arr"):
            if len(out) != len(tensors) or any(
                    o.numel() != g.numel() or o.dtype != torch.float32 or not o.is_contiguous()
                    for o, g in zip(out, tensors.grads.buffers)):
                raise ValueError(f"{name}: expected contiguous fp32 tensors of the list's sizes")
        elif len(out) != len(tensors):
            raise ValueError(f"{name}: expected {len(tensors)} buffers")
        arrays.append(_ptrs(out))
    rc = _lib.zero_adamw_state_f32(len(tensors), tensors.arr, *arrays, _stream_handle(stream))
    if rc != ZERO_OK:
        raise ZeroError(rc, "zero_adamw_state_f32")


__all__ = ["zero_linear_forward", "zero_linear_backward", "zero_linear_workspace", "grad_list",
           "GradList", "grad_norm_workspace", "zero_grad_norm", "adamw_tensors", "AdamwTensors",
           "zero_adamw_step", "zero_adamw_state_f32", "ZeroLinear", "ZeroAdamwTensor"]
