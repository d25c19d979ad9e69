"""The training-step entry points refuse bad arguments with the documented codes before any
CUDA call (no GPU needed; the addresses are never touched)."""
import ctypes

import pytest

import zero_partitioned_mixed_adam_gb300 as za

BASE = 1 << 40
GIB = 1 << 30
CODES = {v: k for k, v in za.ERRORS.items()}
LIB = za.raw_lib()


def at(i):
    return BASE + i * GIB


def shape(rows=64, k=128, out=96, **ld):
    d = dict(ldx=k, ldw=k, ldy=out, ldr=out, ldp=out, ldpi=k, lddx=k, lddw=k)
    d.update(ld)
    return za.ZeroLinear(rows, k, out, *d.values())


def forward(s=None, x=at(1), w=at(2), bias=at(3), act=1, res=at(4), pre=at(5), y=at(6), ws=at(9),
            nbytes=GIB):
    s = shape() if s is None else s
    return LIB.zero_linear_forward(ctypes.byref(s) if s else None, x, w, bias, act, res, pre, y, ws,
                                   nbytes, None)


def test_forward_refusals():
    assert forward(s=0) == CODES["ZERO_E_NULLPTR"]
    for s in (shape(rows=-1), shape(k=0), shape(out=0), shape(k=2 ** 31), shape(ldx=127),
              shape(ldw=100), shape(ldy=95), shape(ldr=1), shape(ldp=0), shape(ldx=2 ** 60)):
        assert forward(s=s) == CODES["ZERO_E_SHAPE"]
    for name in ("x", "w", "y"):
        assert forward(**{name: None}) == CODES["ZERO_E_NULLPTR"]
    assert forward(act=4) == forward(act=-1) == CODES["ZERO_E_LAYOUT"]
    for name in ("x", "w", "bias", "res", "pre", "y"):
        assert forward(**{name: at(7) + 1}) == CODES["ZERO_E_ALIGN"]
    for other in (at(1), at(2) + 2 * 128 * 95, at(3), at(5) + 2):
        assert forward(y=other) == CODES["ZERO_E_ALIAS"]
    assert forward(y=at(4), s=shape(ldy=100, ldr=96)) == CODES["ZERO_E_ALIAS"]  # another pitch
    assert forward(pre=at(4)) == CODES["ZERO_E_ALIAS"]
    # no rows: nothing to do, whatever the epilogue
    s = shape(rows=0)
    assert LIB.zero_linear_forward(ctypes.byref(s), at(1), at(2), None, 0, None, None, at(6), at(9),
                                   GIB, None) == 0


def backward(s=None, dy=at(1), x=at(2), w=at(3), act=2, pre=at(4), act_in=3, pre_in=at(5), dx=at(6),
             dw=at(7), db=at(8), flags=0x50, ws=at(9), nbytes=GIB):
    s = shape() if s is None else s
    return LIB.zero_linear_backward(ctypes.byref(s) if s else None, dy, x, w, act, pre, act_in,
                                    pre_in, dx, dw, db, flags, ws, nbytes, None)


def test_backward_refusals():
    assert backward(s=0) == CODES["ZERO_E_NULLPTR"]
    for s in (shape(rows=-1), shape(k=0), shape(ldy=95), shape(ldx=1), shape(ldw=1), shape(ldp=1),
              shape(ldpi=1), shape(lddx=1), shape(lddw=127)):
        assert backward(s=s) == CODES["ZERO_E_SHAPE"]
    for name in ("dy", "x", "w", "pre", "pre_in"):
        assert backward(**{name: None}) == CODES["ZERO_E_NULLPTR"]
    for kw in (dict(act=4), dict(act_in=-1), dict(flags=0x20), dict(flags=0x80)):
        assert backward(**kw) == CODES["ZERO_E_LAYOUT"]
    for name in ("dy", "x", "w", "pre", "pre_in", "dx"):
        assert backward(**{name: at(10) + 1}) == CODES["ZERO_E_ALIGN"]
    for name in ("dw", "db"):
        assert backward(**{name: at(10) + 2}) == CODES["ZERO_E_ALIGN"]   # fp32 gradients
    assert backward(dx=at(2)) == CODES["ZERO_E_ALIAS"]
    assert backward(dw=at(3) + 400) == CODES["ZERO_E_ALIAS"]
    assert backward(db=at(6)) == CODES["ZERO_E_ALIAS"]
    assert backward(ws=None) == CODES["ZERO_E_WORKSPACE"]
    assert backward(ws=at(9) + 8) == CODES["ZERO_E_WORKSPACE"]
    need = za.zero_linear_workspace(64, 128, 96, True, aligned=True)
    assert need > 0 and backward(nbytes=need - 1) == CODES["ZERO_E_WORKSPACE"]
    most = za.zero_linear_workspace(64, 128, 96, True)
    assert most > need and backward(dy=at(1) + 2, nbytes=most - 1) == CODES["ZERO_E_WORKSPACE"]
    assert LIB.zero_linear_workspace(ctypes.byref(shape()), 8) == CODES["ZERO_E_LAYOUT"]
    assert backward(ws=at(7)) == CODES["ZERO_E_ALIAS"]
    with pytest.raises(za.ZeroError) as e:
        za.zero_linear_workspace(1, 0, 1)
    assert e.value.code == "ZERO_E_SHAPE"


def norm(n=2, grads=(at(1), at(2)), numels=(100, 50), flags=0, most=1.0, out=at(3), ws=at(4),
         nbytes=GIB):
    g = (ctypes.c_void_p * len(grads))(*grads) if grads else None
    k = (ctypes.c_int64 * len(numels))(*numels) if numels else None
    return LIB.zero_grad_norm(n, g, k, flags, most, out, ws, nbytes, None)


def test_norm_refusals():
    assert norm(n=-1) == norm(n=za.ZERO_MAX_LIST + 1) == CODES["ZERO_E_SHAPE"]
    assert norm(numels=(100, -1)) == CODES["ZERO_E_SHAPE"]
    assert norm(flags=0x80) == CODES["ZERO_E_LAYOUT"]
    assert norm(most=-1.0) == norm(most=float("nan")) == norm(most=float("inf")) == CODES["ZERO_E_HPARAM"]
    assert norm(grads=None) == norm(numels=None) == norm(out=None) == CODES["ZERO_E_NULLPTR"]
    assert norm(grads=(at(1), None)) == CODES["ZERO_E_NULLPTR"]
    assert norm(grads=(at(1), at(2) + 1)) == CODES["ZERO_E_ALIGN"]
    assert norm(grads=(at(1), at(2) + 2), flags=0x10) == CODES["ZERO_E_ALIGN"]
    assert norm(out=at(3) + 2) == CODES["ZERO_E_ALIGN"]
    for kw in (dict(ws=None), dict(ws=at(4) + 8), dict(nbytes=LIB.zero_grad_norm_workspace() - 1)):
        assert norm(**kw) == CODES["ZERO_E_WORKSPACE"]
    assert norm(out=at(1) + 196) == norm(out=at(4)) == norm(ws=at(2)) == CODES["ZERO_E_ALIAS"]


def adamw(numel=1000, flags=0x80, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, t=1, scale=None, n=1,
          decay=0.1, **p):
    d = dict(grad=at(1), master=at(2), param_bf16=at(3), m=at(4), v=at(5), m_scale=at(6),
             v_scale=at(7))
    d.update(p)
    arr = (za.ZeroAdamwTensor * 1)(za.ZeroAdamwTensor(numel, *d.values(), decay))
    return LIB.zero_adamw_step(n, arr, flags, lr, b1, b2, eps, t, scale, 1, None)


def test_adamw_refusals():
    assert adamw(n=-1) == adamw(n=za.ZERO_MAX_LIST + 1) == adamw(numel=-1) == CODES["ZERO_E_SHAPE"]
    assert adamw(numel=2 ** 41) == CODES["ZERO_E_SHAPE"]
    assert adamw(flags=0x40) == adamw(flags=0x20) == CODES["ZERO_E_LAYOUT"]
    for kw in (dict(lr=-1.0), dict(lr=float("nan")), dict(b1=1.0), dict(b2=-0.1),
               dict(eps=float("inf")), dict(decay=-0.1), dict(decay=float("nan"))):
        assert adamw(**kw) == CODES["ZERO_E_HPARAM"]
    assert adamw(t=0) == CODES["ZERO_E_STEP"]
    for name in ("grad", "master", "m", "v", "m_scale", "v_scale"):
        assert adamw(**{name: None}) == CODES["ZERO_E_NULLPTR"]
    for name in ("grad", "param_bf16"):
        assert adamw(**{name: at(8) + 1}) == CODES["ZERO_E_ALIGN"]
    for name in ("master", "m_scale", "v_scale"):
        assert adamw(**{name: at(8) + 2}) == CODES["ZERO_E_ALIGN"]
    assert adamw(flags=0, m=at(8) + 2) == CODES["ZERO_E_ALIGN"]
    assert adamw(scale=at(8) + 2) == CODES["ZERO_E_ALIGN"]
    assert adamw(m=at(2) + 8) == adamw(grad=at(5)) == adamw(m_scale=at(6), v_scale=at(6)) == CODES["ZERO_E_ALIAS"]
    assert adamw(scale=at(2)) == CODES["ZERO_E_ALIAS"]
    assert LIB.zero_adamw_step(1, None, 0, 1e-3, .9, .999, 1e-8, 1, None, 0, None) == CODES["ZERO_E_NULLPTR"]
    # nothing to step: no CUDA call, no error
    assert adamw(numel=0, grad=None) == adamw(n=0) == 0


def test_moments_refusals():
    arr = (za.ZeroAdamwTensor * 1)(za.ZeroAdamwTensor(1000, 0, 0, 0, at(4), at(5), at(6), at(7), 0.0))

    def call(m=at(1), v=at(2), n=1, a=arr):
        return LIB.zero_adamw_state_f32(n, a, (ctypes.c_void_p * 1)(m), (ctypes.c_void_p * 1)(v), None)

    assert call(n=-1) == CODES["ZERO_E_SHAPE"]
    assert call(a=None) == call(m=None) == CODES["ZERO_E_NULLPTR"]
    assert call(m=at(1) + 2) == CODES["ZERO_E_ALIGN"]
    assert call(m=at(2) + 100) == call(v=at(4)) == call(v=at(7)) == CODES["ZERO_E_ALIAS"]
    assert LIB.zero_adamw_state_f32(1, arr, None, None, None) == 0


def test_binding_refusals():
    import torch
    bf, f32 = torch.bfloat16, torch.float32
    x, w, y = torch.zeros(4, 8, dtype=bf), torch.zeros(6, 8, dtype=bf), torch.zeros(4, 6, dtype=bf)
    for bad in (dict(x=x.float()), dict(w=torch.zeros(6, 7, dtype=bf)), dict(y=y.t()),
                dict(x=torch.zeros(8, 4, dtype=bf).t()), dict(bias=torch.zeros(5, dtype=bf)),
                dict(residual=torch.zeros(4, 5, dtype=bf)), dict(pre=y.float())):
        kw = dict(x=x, w=w, y=y)
        kw.update(bad)
        with pytest.raises(ValueError):
            za.zero_linear_forward(kw.pop("x"), kw.pop("w"), kw.pop("y"), **kw)
    with pytest.raises(ValueError):
        za.zero_linear_backward(y, None, w, dw=torch.zeros(6, 8))
    with pytest.raises(ValueError):
        za.zero_linear_backward(y, x, w, dw=torch.zeros(6, 8), dbias=torch.zeros(6, dtype=bf))
    g = [torch.zeros(300, dtype=bf)]
    s = [torch.zeros(300)]
    with pytest.raises(ValueError):
        za.grad_list([torch.zeros(3), torch.zeros(3, dtype=bf)])
    with pytest.raises(ValueError):
        za.grad_list([torch.zeros(4, 4, dtype=bf).t()])
    with pytest.raises(ValueError):
        za.adamw_tensors(g, s, s, [torch.zeros(299)])
    with pytest.raises(ValueError):
        za.adamw_tensors(g, s, s, s, m_scale=[torch.zeros(2)])
    code = [torch.zeros(300, dtype=torch.uint8)]
    with pytest.raises(ValueError):
        za.adamw_tensors(g, s, code, code, m_scale=[torch.zeros(1)], v_scale=[torch.zeros(2)])
    lst = za.adamw_tensors(g, s, code, code, m_scale=[torch.zeros(2)], v_scale=[torch.zeros(2)],
                           weight_decay=0.1)
    assert lst.flags == za.ZERO_STATE_8BIT and len(lst) == 1
    with pytest.raises(ValueError):
        za.zero_adamw_state_f32(lst, [torch.zeros(300, dtype=f32)[:299]], None)
    with pytest.raises(ValueError):
        za.zero_adamw_state_f32(za.adamw_tensors(g, s, s, s), s, s)


def test_side_by_side_columns_are_no_overlap():
    """y may be other columns of the buffer x lies in (no rows: nothing is launched)."""
    s = shape(rows=64, k=32, out=32, ldx=96, ldy=96, ldw=32)
    codes = []
    for col in (32, 64, 16):
        codes.append(LIB.zero_linear_forward(ctypes.byref(s), at(1), at(2), None, 9, None, None,
                                             at(1) + 2 * col, at(9), GIB, None))
    assert codes == [CODES["ZERO_E_LAYOUT"]] * 3     # an unknown act is found first
    s.ldr = 96
    # the residual as another pair of columns: only the overlapping one is refused
    assert LIB.zero_linear_forward(ctypes.byref(s), at(1), at(2), None, 0, None, None,
                                   at(1) + 2 * 16, at(9), GIB, None) == CODES["ZERO_E_ALIAS"]


def test_messages_name_what_these_calls_refuse():
    """The statuses are shared with the ZeRO step and the gathers; so are their messages."""
    for code, words in (("ZERO_E_SHAPE", ("pitch", "count", "size")), ("ZERO_E_HPARAM", ("weight_decay", "max_norm", "betas")),
                        ("ZERO_E_LAYOUT", ("activation", "flag", "layout"))):
        assert all(w in za.strerror(CODES[code]) for w in words)
