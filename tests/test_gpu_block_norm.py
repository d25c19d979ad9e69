"""The norms around a block, its gate and residual scale on the GPU against 64 bits."""
import itertools

import pytest
import torch

import model_oracle as o
import zero_partitioned_mixed_adam_gb300 as za

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
KINDS = {"none": za.ZERO_NORM_NONE, "rms": za.ZERO_NORM_RMS, "layer": za.ZERO_NORM_LAYER}
EPS = 1e-5

# rows, width: ones; around a warp's and a block's columns; odd; the widest
SHAPES = [(1, 1), (1, 4096), (2, 8), (5, 33), (37, 255), (64, 256), (9, 257), (130, 768), (1003, 775),
          (17, 1024), (40, 1032), (33, 2048), (700, 4100), (3, 8200), (2, 16385), (2, 32768), (3, 32761)]


def matrix(rows, cols, sigma, seed, pitch=0, offset=0, mean=0.0):
    gen = torch.Generator("cuda").manual_seed(seed)
    flat = torch.empty(offset + rows * (cols + pitch), device="cuda").normal_(mean, sigma, generator=gen).to(BF)
    return flat[offset:].view(rows, cols + pitch)[:, :cols]


def blank(rows, cols, dtype=BF, pitch=0, offset=0):
    flat = torch.full((offset + rows * (cols + pitch),), 7.0, dtype=dtype, device="cuda")
    return flat[offset:].view(rows, cols + pitch)[:, :cols]


def vector(n, sigma, seed, offset=0, mean=0.0):
    return matrix(1, n, sigma, seed, 0, offset, mean)[0]


class Block:
    """One block's inputs, and its outputs in 64 bits with their gradients."""

    def __init__(self, m, d, post, gate, kind, plain=False, pitch=0, offset=0, alpha=0.5):
        self.m, self.d, self.post, self.kind, self.alpha = m, d, post, kind, alpha
        at = dict(pitch=pitch, offset=offset)
        self.at = at
        self.r, self.h = matrix(m, d, 2.0, 1, **at, mean=0.5), matrix(m, d, 1.0, 2, **at, mean=-0.5)
        self.gate = {"none": None, "vector": vector(d, 0.5, 3, offset, 1.0),
                     "matrix": matrix(m, d, 0.5, 4, **at, mean=1.0)}[gate]
        self.w1 = None if post == "none" or plain else vector(d, 0.2, 5, offset, 1.0)
        self.b1 = None if post != "layer" or plain else vector(d, 0.2, 6, offset)
        self.w = None if plain else vector(d, 0.2, 7, offset, 1.0)
        self.b = None if kind != "layer" or plain else vector(d, 0.2, 8, offset)
        self.args = dict(h=self.h, post=KINDS[post], post_weight=self.w1, post_bias=self.b1, gate=self.gate,
                         alpha=alpha, kind=KINDS[kind], weight=self.w, eps=EPS)

    def exact(self, s=None, dy=None, ds=None):
        """(s, y), or the gradients by autograd in 64 bits at the bf16 sum s that the backward
        pass is given."""
        leaves = {n: None if t is None else t.to(F64).requires_grad_()
                  for n, t in (("r", self.r), ("h", self.h), ("w1", self.w1), ("b1", self.b1), ("gate", self.gate),
                               ("w", self.w), ("b", self.b))}
        q = leaves
        s64, y = o.block_norm(q["r"], q["h"], self.post, q["w1"], q["b1"], q["gate"], self.alpha, self.kind, q["w"],
                              q["b"], EPS)
        if dy is None:
            return s64.detach(), y.detach()
        at = s.to(F64).requires_grad_()
        y = o.standardized(at, self.kind, EPS)[0]
        y = y if q["w"] is None else y * q["w"]
        y = y if q["b"] is None else y + q["b"]
        y.backward(dy.to(F64))
        dr = at.grad if ds is None else at.grad + ds.to(F64)
        s64.backward(dr)
        return dr, {n: None if t is None else t.grad for n, t in leaves.items()}


def near(got, want, tol, what):
    assert torch.isfinite(got).all(), what
    bad = (got.to(F64) - want).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), float(((got.to(F64) - want).abs() - tol).max()))


def sum_error(d):
    """A row's sum: 8 columns a vector, up to 8 vectors a thread, a warp's 5 additions and 16
    warps', each 2^-24."""
    return (64 + 5 + 16) * 2.0 ** -24


def check_forward(b, in_place=False):
    m, d = b.m, b.d
    want_s, want_y = b.exact()
    s = b.r.clone() if in_place else blank(m, d, **b.at)
    y = blank(m, d, **b.at)
    za.zero_block_norm_forward(s if in_place else b.r, y, s=s, bias=b.b, **b.args)
    half = 2.0 ** -8
    e = sum_error(d) + 2.0 ** -20          # a norm's relative error: its sums, the root, 8 operations
    # P(h) of size p within e of the largest magnitudes that make it: x - mean is off by e of |x|
    h64 = b.h.to(F64)
    p_size = h64.abs()
    if b.post != "none":
        _, root = o.standardized(h64, b.post, EPS)
        p_size = (h64.abs() + h64.abs().mean(1, keepdim=True)) / root
        p_size = p_size if b.w1 is None else p_size * b.w1.to(F64).abs()
        p_size = p_size if b.b1 is None else p_size + b.b1.to(F64).abs()
    g = 1.0 if b.gate is None else b.gate.to(F64).abs()
    es = abs(b.alpha) * g * p_size * e + 2.0 ** -22 * (want_s.abs() + b.r.to(F64).abs())
    near(s, want_s, es + half * (want_s.abs() + es), "s")
    _, root = o.standardized(want_s, b.kind, EPS)
    w = 1.0 if b.w is None else b.w.to(F64).abs()
    size = want_s.abs() + want_s.abs().mean(1, keepdim=True)
    spread = es + es.mean(1, keepdim=True) + size * (es * size).mean(1, keepdim=True) / root ** 2
    ey = (size * e + spread) / root * w + 2.0 ** -22 * want_y.abs()
    near(y, want_y, ey + half * (want_y.abs() + ey), "y")
    return s, y


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("post,gate,kind", [("none", "none", "rms"), ("rms", "vector", "rms"),
                                            ("layer", "matrix", "layer"), ("none", "vector", "layer"),
                                            ("rms", "none", "layer")])
def test_forward(shape, post, gate, kind):
    check_forward(Block(*shape, post, gate, kind))


@pytest.mark.parametrize("shape", [(37, 256), (130, 775), (20, 2304)])
@pytest.mark.parametrize("pitch,offset", [(8, 8), (8, 1), (1, 0), (5, 3)])
def test_forward_layouts(shape, pitch, offset):
    b = Block(*shape, "layer", "matrix", "layer", pitch=pitch, offset=offset)
    s, y = check_forward(b)
    for view in (s, y):
        flat = view._base
        view.fill_(7.0)
        assert (flat == 7.0).all()


def test_forward_without_weights_and_in_place():
    for post, gate, kind in itertools.product(("none", "rms", "layer"), ("none", "vector"), ("rms", "layer")):
        check_forward(Block(50, 328, post, gate, kind, plain=True), in_place=True)


def test_forward_of_the_first_block():
    """No block before: y is r's norm, s is r; or neither s nor a copy of it is written."""
    b = Block(60, 768, "none", "none", "rms")
    y, s, z = blank(60, 768), blank(60, 768), blank(60, 768)
    za.zero_block_norm_forward(b.r, y, weight=b.w, eps=EPS)
    za.zero_block_norm_forward(b.r, z, s=s, weight=b.w, eps=EPS)
    assert torch.equal(y, z) and torch.equal(s, b.r)
    r64 = b.r.to(F64)
    want = o.standardized(r64, "rms", EPS)[0] * b.w.to(F64)
    near(y, want, (2.0 ** -8 + 2.0 ** -17) * want.abs(), "y")


def check_backward(b, *, dtype=BF, add=False, has_ds=True, in_place=False, want=None):
    m, d = b.m, b.d
    s = b.exact()[0].to(BF)
    if b.at["pitch"] or b.at["offset"]:
        s = blank(m, d, **b.at).copy_(s)
    dy, ds = matrix(m, d, 1.0, 11, **b.at), matrix(m, d, 1.0, 12, **b.at) if has_ds else None
    dr64, grads = b.exact(s, dy, ds)
    mags = magnitudes(b, s, dy, ds)
    out = {"dr": ds.clone() if in_place else blank(m, d, **b.at), "dh": blank(m, d, **b.at)}
    if in_place:
        ds = out["dr"]
    gate_rows = b.gate is not None and b.gate.dim() == 2
    vectors = {"dpost_weight": "w1", "dpost_bias": "b1", "dweight": "w", "dbias": "b"}
    if b.gate is not None:
        if gate_rows:
            out["dgate"] = blank(m, d, **b.at)
        else:
            vectors["dgate"] = "gate"
    before = {}
    for name, of in vectors.items():
        if getattr(b, of) is not None:
            out[name] = vector(d, 1.0, 20 + len(name)).to(dtype) if add else torch.full((d,), 7.0, dtype=dtype, device="cuda")
            before[name] = out[name].to(F64) if add else 0.0
    if want is not None:
        out = {n: t for n, t in out.items() if n in want}
    za.zero_block_norm_backward(dy, s, ds=ds, accumulate=add, **b.args, **out)
    e = 8 * sum_error(d) + 2.0 ** -18
    half = 2.0 ** -8
    for name, exact, mag in (("dr", dr64, mags["dr"]), ("dh", grads["h"], mags["dh"])) + \
            ((("dgate", grads["gate"], mags["gate"]),) if gate_rows else ()):
        if name in out:
            near(out[name], exact, e * mag + half * (exact.abs() + e * mag) + 1e-30, name)
    # sums over rows: up to m/152 + 2 a block, up to 2,432 blocks in 32 runs
    es = e + (m / 152 + 2 + 2432 / 32 + 32) * 2.0 ** -24
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -23
    for name, of in vectors.items():
        if name in out:
            exact = grads[of] + before[name]
            tol = es * mags[of] + 2.0 ** -23 * abs(before[name])
            near(out[name], exact, tol + half * (exact.abs() + tol) + 1e-30, name)
    assert za.device_status() == za.ZERO_OK
    return out


def magnitudes(b, s, dy, ds):
    """The sums of magnitudes that each gradient is made of: what a relative error of every step
    may come to."""
    s, dy = s.to(F64), dy.to(F64).abs()
    w = 1.0 if b.w is None else b.w.to(F64).abs()
    _, root = o.standardized(s, b.kind, EPS)
    xh = (s.abs() + s.abs().mean(1, keepdim=True)) / root
    u = dy * w
    mean = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    dr = (u + mean(u) + xh * mean(u * xh)) / root + (0.0 if ds is None else ds.to(F64).abs())
    out = {"dr": dr, "w": (dy * xh).sum(0), "b": dy.sum(0)}
    h = b.h.to(F64)
    dp = abs(b.alpha) * dr
    hh, root1 = h.abs(), 1.0
    if b.post != "none":
        _, root1 = o.standardized(h, b.post, EPS)
        hh = (h.abs() + mean(h.abs())) / root1
    p = hh if b.w1 is None else hh * b.w1.to(F64).abs()
    p = p if b.b1 is None else p + b.b1.to(F64).abs()
    gate = dp * p
    out["gate"] = gate if b.gate is not None and b.gate.dim() == 2 else gate.sum(0)
    dp = dp if b.gate is None else dp * b.gate.to(F64).abs()
    out["w1"], out["b1"], out["dh"] = (dp * hh).sum(0), dp.sum(0), dp
    if b.post != "none":
        v = dp if b.w1 is None else dp * b.w1.to(F64).abs()
        out["dh"] = (v + mean(v) + hh * mean(v * hh)) / root1
    return out


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("post,gate,kind,dtype,add", [
    ("none", "none", "rms", BF, False), ("rms", "vector", "rms", F32, False), ("layer", "matrix", "layer", F32, True),
    ("none", "vector", "layer", BF, True), ("rms", "none", "layer", BF, False)])
def test_backward(shape, post, gate, kind, dtype, add):
    check_backward(Block(*shape, post, gate, kind), dtype=dtype, add=add)


@pytest.mark.parametrize("post,gate,kind", list(itertools.product(
    ("none", "rms", "layer"), ("none", "vector", "matrix"), ("rms", "layer"))))
def test_backward_without_weights(post, gate, kind):
    check_backward(Block(50, 331, post, gate, kind, plain=True), has_ds=False)
    check_backward(Block(9, 328, post, gate, kind, plain=True), in_place=True)


@pytest.mark.parametrize("shape", [(37, 256), (130, 775), (20, 2304)])
@pytest.mark.parametrize("pitch,offset", [(8, 8), (8, 1), (1, 0), (5, 3)])
def test_backward_layouts(shape, pitch, offset):
    out = check_backward(Block(*shape, "layer", "matrix", "layer", pitch=pitch, offset=offset))
    for name in ("dr", "dh", "dgate"):
        flat = out[name]._base
        out[name].fill_(7.0)
        assert (flat == 7.0).all()


def test_each_gradient_alone():
    for post, gate in (("layer", "vector"), ("rms", "matrix"), ("none", "none")):
        b = Block(70, 520, post, gate, "layer")
        whole = check_backward(b)
        for name, want in whole.items():
            assert torch.equal(check_backward(b, want=(name,))[name], want), name


def test_many_rows():
    check_backward(Block(5000, 64, "rms", "vector", "layer"), dtype=F32)
    check_forward(Block(70000, 16, "rms", "vector", "rms"))


def test_rows_do_not_meet():
    """A row of NaN or infinities leaves the others' outputs alone."""
    b = Block(40, 776, "rms", "matrix", "rms")
    s, y = check_forward(b)
    b.h[7], b.r[9, 5] = float("nan"), float("inf")
    t, z = blank(40, 776), blank(40, 776)
    za.zero_block_norm_forward(b.r, z, s=t, **b.args)
    others = [i for i in range(40) if i not in (7, 9)]
    assert torch.equal(t[others], s[others]) and torch.equal(z[others], y[others])
    assert z[7].isnan().all() and not torch.isfinite(z[9]).all()


def test_rows_of_zeros():
    """eps alone under the root: zeros, and gradients of 1/sqrt(eps)."""
    b = Block(4, 64, "none", "none", "rms")
    b.r.zero_(), b.h.zero_()
    y = blank(4, 64)
    za.zero_block_norm_forward(b.r, y, **b.args)
    assert not y.any()
    check_backward(b)


def test_no_rows():
    none, w = blank(1, 48)[:0], vector(48, 1.0, 1)
    za.zero_block_norm_forward(none, none.clone(), h=none, weight=w)
    dw = torch.full((48,), 7.0, device="cuda")
    za.zero_block_norm_backward(none, none, dweight=dw, accumulate=True)
    assert (dw == 7.0).all()
    za.zero_block_norm_backward(none, none, dr=none.clone(), dweight=dw)
    assert not dw.any()


def test_streams_and_graphs():
    b = Block(300, 1032, "layer", "vector", "layer")
    s, y = check_forward(b)
    dy, ds = matrix(300, 1032, 1.0, 11), matrix(300, 1032, 1.0, 12)

    def eager():    # of the library's own s, which a graph's backward pass takes too
        out = {n: torch.full_like(g, 7.0) for n, g in grads.items()}
        za.zero_block_norm_backward(dy, s, ds=ds, **b.args, **out)
        return out

    grads = check_backward(b)
    grads = eager()
    side = torch.cuda.Stream()
    t, z = blank(300, 1032), blank(300, 1032)
    again = {n: torch.full_like(g, 7.0) for n, g in grads.items()}
    ws = torch.empty(za.zero_block_norm_workspace(300, 1032), dtype=torch.uint8, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    za.zero_block_norm_forward(b.r, z, s=t, bias=b.b, stream=side, **b.args)
    za.zero_block_norm_backward(dy, t, ds=ds, workspace=ws, stream=side, **b.args, **again)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(t, s) and torch.equal(z, y)
    assert all(torch.equal(again[n], grads[n]) for n in grads)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        za.zero_block_norm_forward(b.r, z, s=t, bias=b.b, **b.args)
        za.zero_block_norm_backward(dy, t, ds=ds, **b.args, **again)
    b.h.mul_(3.0)
    graph.replay()
    s, y = check_forward(b)
    assert torch.equal(t, s) and torch.equal(z, y)
    grads = eager()
    assert all(torch.equal(again[n], grads[n]) for n in grads)


def test_gradients_against_differences():
    """dr and dh against central differences of the 64-bit forward pass."""
    b = Block(3, 24, "layer", "vector", "rms")
    dy = matrix(3, 24, 1.0, 11)
    s = b.exact()[0].to(BF)
    dr, dh = blank(3, 24), blank(3, 24)
    za.zero_block_norm_backward(dy, s, dr=dr, dh=dh, **b.args)
    vectors = [None if t is None else t.to(F64) for t in (b.w1, b.b1, b.gate, b.w)]

    def value(r, h):
        w1, b1, gate, w = vectors
        y = o.block_norm(r, h, b.post, w1, b1, gate, b.alpha, b.kind, w, None, EPS)[1]
        return (y * dy.to(F64)).sum()

    pair, step = [b.r.to(F64), b.h.to(F64)], 1e-5
    for which, grad in ((0, dr), (1, dh)):
        for i, j in ((0, 0), (1, 11), (2, 23)):
            moved = []
            for sign in (1, -1):
                at = [t.clone() for t in pair]
                at[which][i, j] += sign * step
                moved.append(value(*at))
            slope = (moved[0] - moved[1]) / (2 * step)
            # s was rounded to bf16 before the backward pass, and the result after it
            assert (grad[i, j].to(F64) - slope).abs() <= 2.0 ** -5 * grad[i].to(F64).abs().max()


@pytest.mark.parametrize("post,kind", [("none", "rms"), ("rms", "rms"), ("layer", "layer")])
def test_rows_of_clusters_do_not_meet(post, kind):
    """Rows that several blocks share: a row of NaN leaves the others' outputs alone, and the same bits
    come every time."""
    m, d = 600, 8208
    b = Block(m, d, post, "vector", kind)
    dy = matrix(m, d, 1.0, 11)

    def run():
        s, y, dr, dh = (blank(m, d) for _ in range(4))
        za.zero_block_norm_forward(b.r, y, s=s, bias=b.b, **b.args)
        za.zero_block_norm_backward(dy, s, dr=dr, dh=dh, **b.args)
        return s, y, dr, dh

    first = run()
    assert all(torch.isfinite(t).all() for t in first)
    for _ in range(10):
        assert all(torch.equal(a, t) for a, t in zip(run(), first))
    b.h[77] = float("nan")
    others = torch.arange(m, device="cuda") != 77
    assert all(torch.equal(a[others], t[others]) and a[77].isnan().any() for a, t in zip(run(), first))


@pytest.mark.parametrize("shape", [(37, 256), (1003, 775), (4096, 2048), (700, 4100), (300, 8200), (64, 32768)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_sums_over_rows_in_fp32(shape, kind):
    """dweight and dbias as near 64 bits as their additions allow, u = 2^-24 each.

    A row's sum of squares: 4 additions of a thread's 8 columns, 5 of lanes, 16 parts of 128 and 3
    of lanes: 28 u, and 2 u for the mean; half of it in the root, 2 ulp (4 u) for rsqrt, 1 u for the
    product: 20 u of x standardized.  LAYER: the mean is off by 30 u of the mean magnitude.  Sums over
    rows: those of a block, its runs of up to 2,432 blocks and 32 runs."""
    m, d = shape
    b = Block(m, d, "none", "none", kind)
    s, dy = matrix(m, d, 2.0, 5, mean=0.5), matrix(m, d, 1.0, 11)
    dw, db = (torch.full((d,), 7.0, device="cuda") for _ in range(2))
    out = dict(dweight=dw, dbias=db) if kind == "layer" else dict(dweight=dw)
    za.zero_block_norm_backward(dy, s, weight=b.w, kind=KINDS[kind], eps=EPS, **out)
    s64, dy64, u = s.to(F64), dy.to(F64), 2.0 ** -24
    standard, root = o.standardized(s64, kind, EPS)
    rows = m / 152 + 2 + 2432 / 32 + 32
    size = (dy64 * standard).abs().sum(0)
    tol = (20 + rows) * u * size
    if kind == "layer":
        off = 30 * u * s64.abs().mean(1, keepdim=True) / root
        tol = tol + (dy64.abs() * (off + u * s64.abs() / root)).sum(0)
        near(db, dy64.sum(0), rows * u * dy64.abs().sum(0), "dbias")
    near(dw, (dy64 * standard).sum(0), tol, "dweight")
