"""The entry points of a model's ends and norms refuse bad arguments with the documented codes
before any CUDA call (no GPU needed; the addresses are never touched), and so does the binding."""
import ctypes

import pytest
import torch

import zero_partitioned_mixed_adam_gb300 as za
from zero_partitioned_mixed_adam_gb300 import model_ops

BASE, GIB = 1 << 40, 1 << 30
CODES = {v: k for k, v in za.ERRORS.items()}
LIB = za.raw_lib()
NAN, INF = float("nan"), float("inf")


def at(i):
    return BASE + i * GIB


def embedding(rows=64, width=128, vocab=1000, ldt=None, ldy=None):
    return za.ZeroEmbedding(rows, width, vocab, width if ldt is None else ldt, width if ldy is None else ldy)


def lookup(s=None, table=at(1), ids=at(2), flags=0, scale=1.0, y=at(3)):
    s = embedding() if s is None else s
    return LIB.zero_embedding_forward(ctypes.byref(s) if s else None, table, ids, flags, scale, y, None)


def scatter(s=None, dy=at(1), ids=at(2), flags=0, scale=1.0, padding=-1, dtable=at(3)):
    s = embedding() if s is None else s
    return LIB.zero_embedding_backward(ctypes.byref(s) if s else None, dy, ids, flags, scale, padding, dtable, None)


@pytest.mark.parametrize("call", [lookup, scatter])
def test_embedding_refusals(call):
    assert call(s=0) == CODES["ZERO_E_NULLPTR"]
    for kw in (dict(rows=-1), dict(width=0), dict(vocab=0), dict(rows=2 ** 31), dict(width=2 ** 31), dict(vocab=2 ** 31),
               dict(ldt=127), dict(ldy=1), dict(ldt=2 ** 60)):
        assert call(s=embedding(**kw)) == CODES["ZERO_E_SHAPE"], kw
    names = ("table", "ids", "y") if call is lookup else ("dy", "ids", "dtable")
    for name in names:
        assert call(**{name: None}) == CODES["ZERO_E_NULLPTR"]
        assert call(**{name: at(9) + 1}) == CODES["ZERO_E_ALIGN"]
    assert call(ids=at(9) + 4) == CODES["ZERO_E_ALIGN"]              # int64
    for flags in (1, 0x20, 0x200) + ((za.ZERO_GRAD_F32,) if call is lookup else (0x80,)):
        assert call(flags=flags) == CODES["ZERO_E_LAYOUT"]
    for scale in (NAN, INF, 1e39):
        assert call(scale=scale) == CODES["ZERO_E_HPARAM"]
    out = names[2]
    assert call(**{out: at(1) + 2 * 64}) == call(**{out: at(2) + 8}) == CODES["ZERO_E_ALIAS"]
    if call is scatter:
        assert call(flags=za.ZERO_GRAD_F32, dtable=at(3) + 2) == CODES["ZERO_E_ALIGN"]
    none = embedding(rows=0)
    assert call(s=none, **({} if call is lookup else dict(flags=za.ZERO_GRAD_ACCUMULATE))) == 0


def ce(rows=64, width=128, vocab=1000, **ld):
    d = dict(ldx=width, ldw=width, lddx=width, lddw=width)
    d.update(ld)
    return za.ZeroCrossEntropy(rows, width, vocab, *d.values())


def loss(s=None, x=at(1), w=at(2), t=at(3), ignore=-100, scale=at(4), losses=at(5), total=at(6), dx=at(7), dw=at(8),
         flags=0, ws=at(9), nbytes=GIB):
    s = ce() if s is None else s
    return LIB.zero_linear_cross_entropy(ctypes.byref(s) if s else None, x, w, t, ignore, scale, losses, total, dx, dw,
                                         flags, ws, nbytes, None)


def test_cross_entropy_refusals():
    assert loss(s=0) == CODES["ZERO_E_NULLPTR"]
    for kw in (dict(rows=-1), dict(width=0), dict(vocab=0), dict(rows=2 ** 31), dict(vocab=2 ** 31), dict(ldx=127),
               dict(ldw=5), dict(lddx=0), dict(lddw=127), dict(ldw=2 ** 60)):
        assert loss(s=ce(**kw)) == CODES["ZERO_E_SHAPE"], kw
    for name in ("x", "w", "t"):
        assert loss(**{name: None}) == CODES["ZERO_E_NULLPTR"]
    for flags in (1, 0x20, 0x80, 0x200):
        assert loss(flags=flags) == CODES["ZERO_E_LAYOUT"]
    for name, off in (("x", 1), ("w", 1), ("t", 4), ("scale", 2), ("losses", 2), ("total", 2), ("dx", 1), ("dw", 1)):
        assert loss(**{name: at(12) + off}) == CODES["ZERO_E_ALIGN"], name
    assert loss(t=at(12) + 4, flags=za.ZERO_IDS_I32, ws=None) == CODES["ZERO_E_WORKSPACE"]
    assert loss(dw=at(12) + 2, flags=za.ZERO_GRAD_F32) == CODES["ZERO_E_ALIGN"]
    outs, ins = ("losses", "total", "dx", "dw"), (at(1), at(2) + 64, at(3), at(4))
    for name in outs:
        for other in ins:
            assert loss(**{name: other}) == CODES["ZERO_E_ALIAS"], (name, other)
    assert loss(dx=at(8) + 512) == loss(losses=at(6)) == CODES["ZERO_E_ALIAS"]
    need = za.zero_linear_cross_entropy_workspace(64, 128, 1000, aligned=True)
    assert loss(nbytes=need - 1) == loss(ws=None) == loss(ws=at(9) + 8) == CODES["ZERO_E_WORKSPACE"]
    most = za.zero_linear_cross_entropy_workspace(64, 128, 1000)
    assert most > need and loss(w=at(2) + 2, nbytes=most - 1) == CODES["ZERO_E_WORKSPACE"]
    alone = za.zero_linear_cross_entropy_workspace(64, 128, 1000, gradients=False, aligned=True)
    assert alone < need and loss(dx=None, dw=None, nbytes=alone - 1) == CODES["ZERO_E_WORKSPACE"]
    assert loss(x=at(9) + 16) == CODES["ZERO_E_ALIAS"]      # the workspace is written
    with pytest.raises(za.ZeroError):
        za.zero_linear_cross_entropy_workspace(1, 0, 1)
    assert LIB.zero_linear_cross_entropy_workspace(None, 0) == CODES["ZERO_E_NULLPTR"]
    assert LIB.zero_linear_cross_entropy_workspace(ctypes.byref(ce()), 4) == CODES["ZERO_E_LAYOUT"]


def test_cross_entropy_workspace_is_bounded_by_the_piece():
    """16 bits of every logit of a piece, not of every row: 1 GiB and what goes with it."""
    one = za.zero_linear_cross_entropy_workspace(8192, 2048, 50257, aligned=True)
    many = za.zero_linear_cross_entropy_workspace(1 << 20, 2048, 50257, f32=True, aligned=True)
    assert one < 2 ** 30 and many < 2.5 * 2 ** 30
    assert za.zero_linear_cross_entropy_workspace(1 << 20, 2048, 50257, gradients=False, aligned=True) < 2 ** 31


def block(rows=64, width=128, post=1, kind=2, alpha=1.0, eps=1e-5, **ld):
    names = ("ldr", "ldh", "ldg", "lds", "ldy", "lddy", "ldds", "lddr", "lddh", "lddg")
    d = {n: 0 if n == "ldg" else width for n in names}
    d.update(ld)
    return za.ZeroBlockNorm(rows, width, post, kind, alpha, eps, *[d[n] for n in names])


def forward(z=None, r=at(1), h=at(2), pw=at(3), pb=None, gate=at(4), w=at(5), b=at(6), s=at(7), y=at(8)):
    z = block() if z is None else z
    return LIB.zero_block_norm_forward(ctypes.byref(z) if z else None, r, h, pw, pb, gate, w, b, s, y, None)


BACK = dict(dy=at(1), ds=at(2), s=at(3), h=at(4), pw=at(5), pb=None, gate=at(6), w=at(7), dr=at(8), dh=at(9), dg=at(10),
            dpw=at(11), dpb=None, dw=at(12), db=at(13))


def backward(z=None, flags=0, ws=at(14), nbytes=GIB, **kw):
    z = block() if z is None else z
    a = {**BACK, **kw}
    return LIB.zero_block_norm_backward(ctypes.byref(z) if z else None, *a.values(), flags, ws, nbytes, None)


SHAPES = [dict(rows=-1), dict(rows=2 ** 31), dict(width=0), dict(width=za.ZERO_MAX_NORM_WIDTH + 1)]
KINDS = [dict(kind=0), dict(kind=3), dict(kind=-1), dict(post=3), dict(post=-1), dict(post=0)]


def test_block_norm_forward_refusals():
    assert forward(z=0) == CODES["ZERO_E_NULLPTR"]
    for kw in SHAPES + [{n: 127} for n in ("ldr", "ldh", "ldg", "lds", "ldy")] + [dict(ldr=2 ** 31)]:
        assert forward(z=block(**kw)) == CODES["ZERO_E_SHAPE"], kw
    for kw in KINDS:      # (post 0: it has no weight)
        assert forward(z=block(**kw)) == CODES["ZERO_E_LAYOUT"], kw
    assert forward(h=None) == forward(z=block(post=0), h=None, pw=None) == CODES["ZERO_E_LAYOUT"]
    assert forward(pb=at(9)) == forward(z=block(kind=1)) == CODES["ZERO_E_LAYOUT"]        # biases are LAYER's
    for kw in (dict(alpha=NAN), dict(alpha=1e39), dict(eps=-1.0), dict(eps=INF), dict(eps=1e39)):
        assert forward(z=block(**kw)) == CODES["ZERO_E_HPARAM"], kw
    for name in ("r", "y"):
        assert forward(**{name: None}) == CODES["ZERO_E_NULLPTR"]
    for name in ("r", "h", "pw", "gate", "w", "b", "s", "y"):
        assert forward(**{name: at(9) + 1}) == CODES["ZERO_E_ALIGN"], name
    for other in (at(1), at(2) + 64, at(3), at(4), at(5), at(6), at(7)):
        assert forward(y=other) == CODES["ZERO_E_ALIAS"]
    for other in (at(2), at(3), at(4), at(5), at(6), at(1) + 2):
        assert forward(s=other) == CODES["ZERO_E_ALIAS"]
    assert forward(s=at(1), z=block(lds=136)) == CODES["ZERO_E_ALIAS"]                     # another pitch
    assert forward(z=block(rows=0)) == 0


def test_block_norm_backward_refusals():
    assert backward(z=0) == CODES["ZERO_E_NULLPTR"]
    for kw in SHAPES + [{n: 127} for n in ("ldh", "ldg", "lds", "lddy", "ldds", "lddr", "lddh")] + [dict(lddr=2 ** 31),
                                                                                                    dict(ldg=128, lddg=1)]:
        assert backward(z=block(**kw)) == CODES["ZERO_E_SHAPE"], kw
    for kw in KINDS:
        assert backward(z=block(**kw)) == CODES["ZERO_E_LAYOUT"], kw
    for kw in (dict(h=None), dict(pb=at(20)), dict(dpb=at(20)), dict(gate=None), dict(flags=1), dict(flags=0x80)):
        assert backward(**kw) == CODES["ZERO_E_LAYOUT"], kw
    assert backward(z=block(kind=1)) == CODES["ZERO_E_LAYOUT"]                             # dbias is LAYER's
    assert backward(z=block(post=0), pw=None) == CODES["ZERO_E_LAYOUT"]                    # and dpost_weight post's
    for name in ("dy", "s"):
        assert backward(**{name: None}) == CODES["ZERO_E_NULLPTR"]
    for name in BACK:
        if BACK[name] is not None:
            assert backward(**{name: at(20) + 1}) == CODES["ZERO_E_ALIGN"], name
    for name in ("dg", "dpw", "dw", "db"):
        assert backward(flags=za.ZERO_GRAD_F32, **{name: at(20) + 2}) == CODES["ZERO_E_ALIGN"], name
    ins, outs = ("dy", "ds", "s", "h", "pw", "gate", "w"), ("dr", "dh", "dg", "dpw", "dw", "db")
    for out in outs:
        for name in ins:
            if (out, name) != ("dr", "ds"):
                assert backward(**{out: BACK[name]}) == CODES["ZERO_E_ALIAS"], (out, name)
        for other in outs:
            if other != out:
                assert backward(**{out: BACK[other]}) == CODES["ZERO_E_ALIAS"], (out, other)
    assert backward(dr=at(2), z=block(lddr=136)) == CODES["ZERO_E_ALIAS"]
    need = za.zero_block_norm_workspace(64, 128)
    assert backward(nbytes=need - 1) == backward(ws=None) == backward(ws=at(14) + 8) == CODES["ZERO_E_WORKSPACE"]
    assert backward(w=at(14) + 16) == CODES["ZERO_E_ALIAS"]
    with pytest.raises(za.ZeroError):
        za.zero_block_norm_workspace(1, 0)
    assert LIB.zero_block_norm_workspace(None) == CODES["ZERO_E_NULLPTR"]


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_the_binding_checks_shapes_types_and_devices():
    ids, t = torch.zeros(4, dtype=torch.int64), torch.zeros(4, dtype=torch.int64)
    m, v, f = bf(4, 8), bf(8), torch.zeros(4)
    table = bf(10, 8)
    bad = [lambda: za.zero_embedding_forward(ids.float(), table, m), lambda: za.zero_embedding_forward(ids, table, bf(4, 7)),
           lambda: za.zero_embedding_forward(ids, table.float(), m), lambda: za.zero_embedding_forward(ids[::2], table, bf(2, 8)),
           lambda: za.zero_embedding_forward(ids.view(2, 2), table, m), lambda: za.zero_embedding_forward(ids, table[0], m),
           lambda: za.zero_embedding_backward(m, ids, table.half()), lambda: za.zero_embedding_backward(m.t(), ids, table),
           lambda: za.zero_linear_cross_entropy(m, table, t[:3]), lambda: za.zero_linear_cross_entropy(m, table, t.float()),
           lambda: za.zero_linear_cross_entropy(m, bf(10, 7), t), lambda: za.zero_linear_cross_entropy(m[0], table, t),
           lambda: za.zero_linear_cross_entropy(m, table, t, f.double()), lambda: za.zero_linear_cross_entropy(m, table, t, f[:3]),
           lambda: za.zero_linear_cross_entropy(m, table, t, f, dx=m.float()), lambda: za.zero_linear_cross_entropy(m, table, t, dw=table.half()),
           lambda: za.zero_linear_cross_entropy(m, table, t, scale=f[:2]),
           lambda: za.zero_block_norm_forward(m, bf(4, 7)), lambda: za.zero_block_norm_forward(m, m.float()),
           lambda: za.zero_block_norm_forward(m, m, h=bf(3, 8)), lambda: za.zero_block_norm_forward(m, m, weight=bf(7)),
           lambda: za.zero_block_norm_forward(m, m, weight=v.float()), lambda: za.zero_block_norm_forward(m, m, weight=bf(16)[::2]),
           lambda: za.zero_block_norm_forward(m, m, h=m, gate=bf(4, 7)), lambda: za.zero_block_norm_forward(v, v),
           lambda: za.zero_block_norm_forward(bf(8, 4).t(), m),
           lambda: za.zero_block_norm_backward(m, m, dweight=v.half()), lambda: za.zero_block_norm_backward(m, m, dweight=v[:7]),
           lambda: za.zero_block_norm_backward(m, m, dweight=v, dbias=v.float()),
           lambda: za.zero_block_norm_backward(m, m, h=m, gate=v, dgate=m), lambda: za.zero_block_norm_backward(m, m, dgate=v),
           lambda: za.zero_block_norm_backward(m, m, dr=bf(4, 8, 1)),
           # and all of them on the host: these calls take tensors of the current device
           lambda: za.zero_embedding_forward(ids, table, m), lambda: za.zero_embedding_backward(m, ids, table),
           lambda: za.zero_linear_cross_entropy(m, table, t, f), lambda: za.zero_block_norm_forward(m, m.clone()),
           lambda: za.zero_block_norm_backward(m, m, dr=m.clone())]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k} went through")


def test_another_device_and_stream(monkeypatch):
    """Tensors of a device that is not the current one, and a stream of another, are refused."""

    class Tensor:
        def __init__(self, device):
            self.device = device

        def get_device(self):
            return self.device

    class Stream:
        device = torch.device("cuda", 1)

    monkeypatch.setattr(model_ops, "_current_device", lambda: 0)
    model_ops._here(None, (Tensor(0), None, Tensor(0)))
    model_ops._here(12345, (Tensor(0),))
    for stream, tensors in ((None, (Tensor(0), Tensor(1))), (None, (Tensor(-1),)), (Stream(), (Tensor(0),))):
        with pytest.raises(ValueError):
            model_ops._here(stream, tensors)


def test_gates_whose_rows_overlap_are_refused(monkeypatch):
    """A matrix gate or dgate of expanded or overlapping rows: as if its rows lay one after the
    other, it would be read and written past its end."""
    called = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: called.append(args[0]._obj) or 0

    monkeypatch.setattr(model_ops, "_here", lambda *args: None)
    monkeypatch.setattr(model_ops, "_stream_handle", lambda stream: None)
    monkeypatch.setattr(model_ops, "_lib", Library())
    m, workspace = bf(4, 8), torch.empty(1, dtype=torch.uint8)
    expanded, overlapping = bf(8).expand(4, 8), bf(32).as_strided((4, 8), (5, 1))
    for gate in (expanded, overlapping):
        with pytest.raises(ValueError, match="gate"):
            za.zero_block_norm_forward(m, m, h=m, gate=gate)
        with pytest.raises(ValueError, match="gate"):
            za.zero_block_norm_backward(m, m, h=m, gate=gate, dgate=m, workspace=workspace)
        with pytest.raises(ValueError, match="dgate"):
            za.zero_block_norm_backward(m, m, h=m, gate=m, dgate=gate, workspace=workspace)
    assert not called
    # one row has any pitch; columns of a wider matrix are read where they lie
    za.zero_block_norm_forward(m[:1], m[:1], h=m[:1], gate=expanded[:1])
    za.zero_block_norm_forward(m, m, h=m, gate=bf(4, 24)[:, 8:16])
    za.zero_block_norm_backward(m, m, h=m, gate=m, dgate=bf(4, 24)[:, 8:16], workspace=workspace)
    assert [s.ldg for s in called] == [8, 24, 8] and called[2].lddg == 24


def test_the_largest_sides():
    """Sides below 2^31 - 1 are taken, and not 2^31 - 1 itself: as the header says."""
    most = 2 ** 31 - 1
    for kw in (dict(rows=most), dict(width=most), dict(vocab=most)):
        assert lookup(s=embedding(**kw)) == scatter(s=embedding(**kw)) == loss(s=ce(**kw)) == CODES["ZERO_E_SHAPE"]
    # (of no rows: checked and done, or refused for the workspace, before any CUDA call)
    for kw in (dict(width=most - 1, vocab=1), dict(vocab=most - 1, width=1)):
        assert lookup(s=embedding(rows=0, **kw)) == 0
        assert loss(s=ce(rows=0, **kw), ws=None) == CODES["ZERO_E_WORKSPACE"]


def test_cross_entropy_workspace_of_more_than_memory_is_refused():
    """Matrices of more elements than a call takes have no workspace, instead of one that wraps."""
    most = 2 ** 31 - 2
    for rows, width, vocab in ((64, most, most), (0, most, most), (most, most, 1), (64, 1 << 30, 1 << 30)):
        for flags in (0, za.ZERO_LINEAR_BACKWARD, za.ZERO_LINEAR_BACKWARD | za.ZERO_GRAD_F32 | za.ZERO_LINEAR_ALIGNED):
            s = ce(rows=rows, width=width, vocab=vocab)
            assert LIB.zero_linear_cross_entropy_workspace(ctypes.byref(s), flags) == CODES["ZERO_E_SHAPE"]
    for rows, width, vocab in ((64, 1 << 29, (1 << 30) - 1), (most, 1, most), (most, 1 << 28, 1)):
        sizes = [za.zero_linear_cross_entropy_workspace(rows, width, vocab, f32=f32) for f32 in (True, False)]
        # at least a copy of w and of a piece of rows
        assert all(2 * (vocab * width + min(rows, 64) * width) <= n < 2 ** 62 for n in sizes)
