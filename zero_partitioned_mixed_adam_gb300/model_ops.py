"""Binding of the two ends of a model and what stands between its blocks: the embedding of
token ids and its gradient, softmax cross entropy of a linear map onto a vocabulary with its
gradients, and the norms before and after a block with its gate and residual scale.

Like the rest of the binding it marshals arguments only; everything here is reached through
the package itself (zero_embedding_forward, zero_linear_cross_entropy, ...).  Unlike the
optimizer's calls these take tensors of the current CUDA device only.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import (ZERO_GRAD_ACCUMULATE, ZERO_GRAD_F32, ZERO_IDS_I32, ZERO_LINEAR_ALIGNED,
               ZERO_LINEAR_BACKWARD, ZERO_NORM_LAYER, ZERO_NORM_NONE, ZERO_NORM_RMS, ZERO_OK,
               ZeroError, _lib, _stream_handle)
from .train_ops import _BF16, _GRADS, _matrix, _vector

_B = torch.bfloat16


class ZeroEmbedding(ctypes.Structure):
    """zero_embedding_t: sizes and row pitches of a table and the rows looked up in it."""

    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "width", "vocab", "ldt", "ldy")]


class ZeroCrossEntropy(ctypes.Structure):
    """zero_cross_entropy_t: sizes and row pitches of a linear map onto a vocabulary."""

    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "width", "vocab", "ldx", "ldw", "lddx", "lddw")]


class ZeroBlockNorm(ctypes.Structure):
    """zero_block_norm_t: sizes, kinds, scalars and row pitches of a block's norms."""

    _fields_ = [("rows", ctypes.c_int64), ("width", ctypes.c_int64), ("post", ctypes.c_int32),
                ("kind", ctypes.c_int32), ("alpha", ctypes.c_double), ("eps", ctypes.c_double)] + [
        (n, ctypes.c_int64) for n in ("ldr", "ldh", "ldg", "lds", "ldy", "lddy", "ldds", "lddr",
                                      "lddh", "lddg")]


def _declare(lib) -> None:
    vp, i32, i64, dbl = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double
    emb, ce, bn = (ctypes.POINTER(t) for t in (ZeroEmbedding, ZeroCrossEntropy, ZeroBlockNorm))
    lib.zero_embedding_forward.argtypes = [emb, vp, vp, i32, dbl, vp, vp]
    lib.zero_embedding_backward.argtypes = [emb, vp, vp, i32, dbl, i64, vp, vp]
    lib.zero_linear_cross_entropy.argtypes = [ce, vp, vp, vp, i64, vp, vp, vp, vp, vp, i32, vp, i64, vp]
    lib.zero_linear_cross_entropy_workspace.argtypes = [ce, i32]
    lib.zero_block_norm_forward.argtypes = [bn] + [vp] * 10
    lib.zero_block_norm_backward.argtypes = [bn] + [vp] * 15 + [i32, vp, i64, vp]
    lib.zero_block_norm_workspace.argtypes = [bn]
    for name in ("zero_embedding_forward", "zero_embedding_backward", "zero_linear_cross_entropy",
                 "zero_block_norm_forward", "zero_block_norm_backward"):
        getattr(lib, name).restype = ctypes.c_int
    for name in ("zero_linear_cross_entropy_workspace", "zero_block_norm_workspace"):
        getattr(lib, name).restype = i64


_declare(_lib)

_IDS = (torch.int64, torch.int32)


_current_device = torch._C._cuda_getDevice  # (of a process that has tensors there)


def _here(stream, tensors):
    """Refuses tensors and streams that are not of the current CUDA device, on which the
    library launches."""
    here = tensors[0].get_device()
    if here < 0 or here != _current_device():
        raise ValueError(f"expected tensors of the current CUDA device, not of {tensors[0].device}")
    for t in tensors:
        if t is not None and t.get_device() != here:
            raise ValueError(f"expected tensors of one device, not of cuda:{here} and {t.device}")
    if stream is not None and not isinstance(stream, int) and stream.device.index != here:
        raise ValueError(f"the tensors are on cuda:{here}, the stream on {stream.device}")


def _rows(name, t, shape):
    """_matrix for bf16, of a shape."""
    if t.shape != shape or t.dtype is not _B:
        _matrix(name, t, *shape)  # (says what is wrong)
    pitch, step = t.stride()
    rows, cols = shape
    if step != 1 and cols > 1:
        _matrix(name, t, rows, cols)
    return pitch if rows > 1 else max(cols, pitch)


def _gate_rows(name, t, shape):
    """_rows, of a matrix that a pitch of 0 would make a vector."""
    pitch = _rows(name, t, shape)
    if pitch < shape[1]:
        raise ValueError(f"{name}: its rows overlap (pitch {pitch}, {shape[1]} columns)")
    return pitch


def _floats(name, t, n):
    """_vector for fp32."""
    if t.shape != (n,) or t.dtype is not torch.float32 or not t.is_contiguous():
        _vector(name, t, n, (torch.float32,))


def _pointer(t):
    return None if t is None else t.data_ptr()


def _columns(name, t, shape):
    """_vector for bf16, of a shape."""
    if t.shape != shape or t.dtype is not _B or not t.is_contiguous():
        _vector(name, t, shape[0])


@functools.lru_cache(maxsize=256)
def _bytes(call, sizes, *flags):
    """Bytes of workspace, which follow from the sizes."""
    need = getattr(_lib, call)(ctypes.byref(sizes[0](*sizes[1:])), *flags)
    if need < 0:
        raise ZeroError(need, call)
    return need


def _workspace(need, device, stream):
    """Memory from PyTorch's allocator, which is asked while the call's stream is current: it
    hands memory out in that stream's order."""
    if stream is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device)
    with torch.cuda.stream(stream):
        return torch.empty(need, dtype=torch.uint8, device=device)


def _check(rc, what):
    if rc != ZERO_OK:
        raise ZeroError(rc, what)


# ---------------------------------------------------------------------- embedding

def _embedding(ids, table, rows, name, kinds):
    if ids.dim() != 1 or ids.dtype not in _IDS or not ids.is_contiguous():
        raise ValueError(f"ids: expected contiguous int64 or int32, got {tuple(ids.shape)} {ids.dtype}")
    if table.dim() != 2:
        raise ValueError(f"{name} is a matrix")
    vocab, width = table.shape
    n = ids.numel()
    s = ZeroEmbedding(n, width, vocab, _matrix(name, table, vocab, width, kinds), _rows("the rows", rows, (n, width)))
    return s, ZERO_IDS_I32 if ids.dtype is torch.int32 else 0


def zero_embedding_forward(ids, table, y, *, scale: float = 1.0, stream=None) -> None:
    """y[i] = scale * table[ids[i]] for ids [rows] (int64 or int32), table [vocab, width] and
    y [rows, width], bf16 with contiguous columns.  Ids outside the table give rows of NaN."""
    s, flags = _embedding(ids, table, y, "table", _BF16)
    _here(stream, (ids, table, y))
    _check(_lib.zero_embedding_forward(ctypes.byref(s), table.data_ptr(), ids.data_ptr(), flags, scale, y.data_ptr(),
                                       _stream_handle(stream)), "zero_embedding_forward")


def zero_embedding_backward(dy, ids, dtable, *, scale: float = 1.0, padding=None,
                            accumulate: bool = False, stream=None) -> None:
    """dtable[v] = scale * (sum of the rows of dy whose id is v), zeros where there are none; or
    with accumulate=True added to dtable.  dy bf16, dtable bf16 or fp32.  Rows whose id is
    `padding`, or outside the table, have no gradient."""
    s, flags = _embedding(ids, dtable, dy, "dtable", _GRADS)
    flags |= ZERO_GRAD_F32 if dtable.dtype == torch.float32 else 0
    flags |= ZERO_GRAD_ACCUMULATE if accumulate else 0
    _here(stream, (dy, ids, dtable))
    _check(_lib.zero_embedding_backward(ctypes.byref(s), dy.data_ptr(), ids.data_ptr(), flags, scale,
                                        -1 if padding is None else padding, dtable.data_ptr(),
                                        _stream_handle(stream)), "zero_embedding_backward")


# ------------------------------------------------------------------ cross entropy

def zero_linear_cross_entropy_workspace(rows: int, width: int, vocab: int, gradients: bool = True,
                                        f32: bool = False, aligned: bool = False) -> int:
    """Bytes of workspace that suffice for a cross entropy of these sizes; gradients: dx or dw
    is wanted; f32: dw is fp32; aligned: w starts on a 16-byte boundary and its pitch is a
    multiple of 8."""
    flags = (ZERO_LINEAR_BACKWARD if gradients else 0) | (ZERO_LINEAR_ALIGNED if aligned else 0) | \
        (ZERO_GRAD_F32 if f32 else 0)
    return _bytes("zero_linear_cross_entropy_workspace", (ZeroCrossEntropy, rows, width, vocab), flags)


def zero_linear_cross_entropy(x, w, targets, losses=None, total=None, *, dx=None, dw=None,
                              ignore_index: int = -100, scale=None, accumulate: bool = False,
                              workspace=None, stream=None) -> None:
    """Softmax cross entropy of z = x w^T against targets, without keeping z:
    losses[i] = logsumexp(z[i]) - z[i, targets[i]], total = sum of c[i] losses[i], and total's
    gradients dx and dw (dw added to with accumulate=True), each where it is given.

    x [rows, width], w [vocab, width], dx: bf16; targets [rows]: int64 or int32; dw bf16 or
    fp32; losses [rows], total [1], scale [rows]: fp32.  c is scale, or 1 / (rows that are not
    ignored).  Rows whose target is ignore_index are ignored: 0 everywhere.  Other targets
    outside [0, vocab) make their loss NaN.  Without a workspace tensor
    (zero_linear_cross_entropy_workspace bytes) one is taken from PyTorch's allocator."""
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x and w are matrices")
    shape, table = x.shape, w.shape
    rows, width = shape
    vocab = table[0]
    if targets.shape != (rows,) or targets.dtype not in _IDS or not targets.is_contiguous():
        raise ValueError(f"targets: expected {rows} contiguous int64 or int32, got "
                         f"{tuple(targets.shape)} {targets.dtype}")
    s = ZeroCrossEntropy(rows, width, vocab, _rows("x", x, shape), _rows("w", w, (vocab, width)))
    if losses is not None:
        _floats("losses", losses, rows)
    if total is not None:
        _floats("total", total, 1)
    if scale is not None:
        _floats("scale", scale, rows)
    flags = ZERO_IDS_I32 if targets.dtype is torch.int32 else 0
    if dx is not None:
        s.lddx = _rows("dx", dx, shape)
    if dw is not None:
        s.lddw = _matrix("dw", dw, vocab, width, _GRADS)
        if dw.dtype is torch.float32:
            flags |= ZERO_GRAD_F32
    if accumulate:
        flags |= ZERO_GRAD_ACCUMULATE
    _here(stream, (x, w, targets, losses, total, scale, dx, dw, workspace))
    at = w.data_ptr()
    if workspace is None:
        kind = (ZERO_LINEAR_BACKWARD if dx is not None or dw is not None else 0) | (flags & ZERO_GRAD_F32)
        if at % 16 == 0 and (vocab == 1 or s.ldw % 8 == 0):
            kind |= ZERO_LINEAR_ALIGNED
        workspace = _workspace(_bytes("zero_linear_cross_entropy_workspace", (ZeroCrossEntropy, rows, width, vocab), kind),
                               x.device, stream)
    _check(_lib.zero_linear_cross_entropy(ctypes.byref(s), x.data_ptr(), at, targets.data_ptr(), ignore_index,
                                          _pointer(scale), _pointer(losses), _pointer(total), _pointer(dx),
                                          _pointer(dw), flags, workspace.data_ptr(),
                                          workspace.numel() * workspace.element_size(), _stream_handle(stream)),
           "zero_linear_cross_entropy")


# -------------------------------------------------------------------- block norms

def _block_norm(shape, post, kind, alpha, eps, h, gate, w1, b1, w):
    """The sizes with the pitches of h and gate; the vectors checked."""
    rows, width = shape
    s = ZeroBlockNorm(rows, width, post, kind, alpha, eps)
    if h is not None:
        s.ldh = _rows("h", h, shape)
    one = (width,)
    if gate is not None:
        if gate.dim() == 1:
            _columns("gate", gate, one)
        else:
            s.ldg = _gate_rows("gate", gate, shape)
    if w1 is not None:
        _columns("post_weight", w1, one)
    if b1 is not None:
        _columns("post_bias", b1, one)
    if w is not None:
        _columns("weight", w, one)
    return s


def zero_block_norm_forward(r, y, *, h=None, s=None, post: int = ZERO_NORM_NONE, post_weight=None,
                            post_bias=None, gate=None, alpha: float = 1.0, kind: int = ZERO_NORM_RMS,
                            weight=None, bias=None, eps: float = 1e-5, stream=None) -> None:
    """s = r + alpha * gate * P(h) and y = N(s), each row by itself, all bf16.

    r, y, h, s [rows, width] with contiguous columns; h None: s is r.  P: the norm `post`
    (ZERO_NORM_NONE, _RMS, _LAYER) with post_weight and post_bias; N: `kind` (RMS or LAYER) with
    weight and bias (vectors; None: 1 and 0).  gate: a vector [width] or a matrix [rows, width].
    s may be r itself, or None where only y is wanted."""
    if r.dim() != 2:
        raise ValueError("r is a matrix")
    shape = r.shape
    z = _block_norm(shape, post, kind, alpha, eps, h, gate, post_weight, post_bias, weight)
    if bias is not None:
        _columns("bias", bias, (shape[1],))
    z.ldr = _rows("r", r, shape)
    z.ldy = _rows("y", y, shape)
    if s is not None:
        z.lds = _rows("s", s, shape)
    _here(stream, (r, y, h, s, post_weight, post_bias, gate, weight, bias))
    _check(_lib.zero_block_norm_forward(ctypes.byref(z), _pointer(r), _pointer(h), _pointer(post_weight),
                                        _pointer(post_bias), _pointer(gate), _pointer(weight), _pointer(bias),
                                        _pointer(s), _pointer(y), _stream_handle(stream)),
           "zero_block_norm_forward")


def zero_block_norm_workspace(rows: int, width: int) -> int:
    """Bytes of workspace that suffice for zero_block_norm_backward."""
    return _bytes("zero_block_norm_workspace", (ZeroBlockNorm, rows, width))


def zero_block_norm_backward(dy, s, *, ds=None, h=None, post: int = ZERO_NORM_NONE, post_weight=None,
                             post_bias=None, gate=None, alpha: float = 1.0, kind: int = ZERO_NORM_RMS,
                             weight=None, eps: float = 1e-5, dr=None, dh=None, dgate=None,
                             dpost_weight=None, dpost_bias=None, dweight=None, dbias=None,
                             accumulate: bool = False, workspace=None, stream=None) -> None:
    """Gradients of zero_block_norm_forward, from dy and the gradient ds that reaches s from
    elsewhere (None: 0); each output that is given is written.

    dr, dh and a matrix dgate are bf16; dpost_weight, dpost_bias, dweight, dbias and a vector
    dgate are bf16 or fp32, all alike, and added to with accumulate=True.  dr may be ds itself."""
    if dy.dim() != 2:
        raise ValueError("dy is a matrix")
    shape = dy.shape
    z = _block_norm(shape, post, kind, alpha, eps, h, gate, post_weight, post_bias, weight)
    z.lddy = _rows("dy", dy, shape)
    z.lds = _rows("s", s, shape)
    if ds is not None:
        z.ldds = _rows("ds", ds, shape)
    if dr is not None:
        z.lddr = _rows("dr", dr, shape)
    if dh is not None:
        z.lddh = _rows("dh", dh, shape)
    vectors = (dpost_weight, dpost_bias, dweight, dbias, dgate)
    if dgate is not None:
        if gate is None or dgate.dim() != gate.dim():
            raise ValueError("dgate is of gate's shape")
        if gate.dim() == 2:
            z.lddg = _gate_rows("dgate", dgate, shape)
            vectors = vectors[:4]
    kind_of = None
    for t in vectors:
        if t is None:
            continue
        if t.shape != (shape[1],) or t.dtype not in _GRADS or not t.is_contiguous():
            _vector("a vector's gradient", t, shape[1], _GRADS)
        if kind_of is not None and t.dtype is not kind_of:
            raise ValueError("the gradients of vectors are bf16 or fp32, all alike")
        kind_of = t.dtype
    flags = (ZERO_GRAD_F32 if kind_of is torch.float32 else 0) | (ZERO_GRAD_ACCUMULATE if accumulate else 0)
    _here(stream, (dy, s, ds, h, post_weight, post_bias, gate, weight, dr, dh, dgate, dpost_weight,
                   dpost_bias, dweight, dbias, workspace))
    if workspace is None:
        workspace = _workspace(_bytes("zero_block_norm_workspace", (ZeroBlockNorm, *shape)), dy.device, stream)
    _check(_lib.zero_block_norm_backward(
        ctypes.byref(z), dy.data_ptr(), _pointer(ds), s.data_ptr(), _pointer(h), _pointer(post_weight),
        _pointer(post_bias), _pointer(gate), _pointer(weight), _pointer(dr), _pointer(dh), _pointer(dgate),
        _pointer(dpost_weight), _pointer(dpost_bias), _pointer(dweight), _pointer(dbias), flags, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_handle(stream)), "zero_block_norm_backward")


__all__ = ["zero_embedding_forward", "zero_embedding_backward", "zero_linear_cross_entropy",
           "zero_linear_cross_entropy_workspace", "zero_block_norm_forward", "zero_block_norm_backward",
           "zero_block_norm_workspace", "ZeroEmbedding", "ZeroCrossEntropy", "ZeroBlockNorm"]
