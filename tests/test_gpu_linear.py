"""Linear maps, forward and backward, on the GPU against products in 64 bits."""
import math

import numpy as np
import pytest
import torch

import train_oracle as o
import zero_partitioned_mixed_adam_gb300 as za

pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def normal(shape, sigma, seed, pitch=0, offset=0):
    """A bf16 matrix; pitch: extra elements between rows; offset: elements before the first."""
    gen = torch.Generator("cuda").manual_seed(seed)
    rows, cols = shape
    flat = torch.empty(offset + rows * (cols + pitch), device="cuda").normal_(0, sigma, generator=gen).to(BF)
    return flat[offset:].view(rows, cols + pitch)[:, :cols]


def empty(shape, dtype=BF, pitch=0, offset=0):
    flat = torch.full((offset + shape[0] * (shape[1] + pitch),), 7.0, dtype=dtype, device="cuda")
    return flat[offset:].view(shape[0], shape[1] + pitch)[:, :shape[1]]


def host(t):
    return t.double().cpu().numpy()


def product_error(a, b, depth):
    """Bound of an fp32 product's error: sums of 16 products or more at a time, each of the
    depth/16 + 2 additions good to 2^-22 of the sum of magnitudes so far."""
    return (depth / 16 + 2) * 2.0 ** -22 * host(a.double().abs() @ b.double().abs())


def check(got, want, tol, what):
    got = host(got)
    assert np.isfinite(got).all(), what
    bad = np.abs(got - want) > tol
    assert not bad.any(), (what, int(bad.sum()), float((np.abs(got - want) - tol).max()))


# sizes: one row and one feature; around the tiles of 16 to 256; odd; longer
SHAPES = [(1, 1, 1), (1, 64, 64), (1, 4096, 1000), (2, 100, 72), (3, 1027, 515), (5, 768, 2304),
          (8, 512, 256), (16, 256, 4096), (17, 130, 70), (31, 2048, 96), (64, 640, 384),
          (65, 192, 136), (127, 128, 129), (128, 128, 256), (129, 64, 257), (255, 72, 264),
          (256, 256, 256), (257, 320, 512), (300, 775, 1031), (777, 768, 2304), (1024, 1024, 1024),
          (2000, 520, 296), (4100, 136, 72)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
def test_forward(shape, act):
    m, k, n = shape
    x, w = normal((m, k), 1.0, 1), normal((n, k), 1.0 / math.sqrt(k), 2)
    bias, res = normal((1, n), 0.5, 3)[0], normal((m, n), 1.0, 4)
    plain = act == "none"
    y, pre = empty((m, n)), empty((m, n))
    za.zero_linear_forward(x, w, y, bias=None if plain else bias, act=o.ACTS[act],
                           residual=None if act == "relu" else res, pre=None if plain else pre)
    z = host(x) @ host(w).T + (0.0 if plain else host(bias))
    ez = product_error(x, w.t(), k) + 2.0 ** -22 * np.abs(z)
    want = o.act(z, act) + (0.0 if act == "relu" else host(res))
    # the sum's error through the slope, the exponential's and the quotients' few ulp, and
    # the one rounding to bf16
    tol = o.SLOPE[act] * ez + 2.0 ** -18 * np.abs(z) + 2.0 ** -8 * np.abs(want) + 1e-30
    check(y, want, tol, "y")
    if not plain:
        check(pre, z, ez + 2.0 ** -8 * np.abs(z) + 1e-30, "pre")


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("act,act_in,dtype,add", [("none", "none", F32, False), ("none", "silu", F32, True),
                                                  ("gelu", "none", BF, False), ("silu", "gelu", BF, True),
                                                  ("relu", "relu", F32, True)])
def test_backward(shape, act, act_in, dtype, add):
    m, k, n = shape
    x, w, dy = normal((m, k), 1.0, 1), normal((n, k), 1.0 / math.sqrt(k), 2), normal((m, n), 1.0, 3)
    pre = normal((m, n), 1.0, 4) if act != "none" else None
    pre_in = normal((m, k), 1.0, 5) if act_in != "none" else None
    dw = normal((n, k), 1.0, 6).to(dtype) if add else empty((n, k), dtype)
    db = normal((1, n), 1.0, 7)[0].to(dtype) if add else empty((1, n), dtype)[0]
    dx, dw0, db0 = empty((m, k)), host(dw), host(db)
    za.zero_linear_backward(dy, x, w, dx=dx, dw=dw, dbias=db, act=o.ACTS[act], pre=pre,
                            act_in=o.ACTS[act_in], pre_in=pre_in, accumulate=add)
    s = np.ones((m, n)) if pre is None else o.slope(host(pre), act)
    dz = host(dy) * s
    adz = torch.from_numpy(np.abs(dz)).cuda()
    # dz as the products take it: the slope's few ulp, then rounded to bf16
    edz = 0.0 if pre is None else 2.0 ** -8
    s_in = np.ones((m, k)) if pre_in is None else o.slope(host(pre_in), act_in)
    want = (dz @ host(w)) * s_in
    tol = (product_error(adz, w, n) + edz * host(adz @ w.double().abs())) * np.abs(s_in)
    tol = tol + 2.0 ** -17 * np.abs(dz @ host(w)) + 2.0 ** -8 * np.abs(want) + 1e-30
    check(dx, want, tol, "dx")
    keep = 1.0 if add else 0.0
    last = 2.0 ** -8 if dtype == BF else 2.0 ** -23
    want = dz.T @ host(x) + keep * dw0
    tol = product_error(adz.t(), x, m) + edz * host(adz.t() @ x.double().abs()) + last * np.abs(want)
    check(dw, want, tol + 2.0 ** -23 * np.abs(keep * dw0) + 1e-30, "dw")
    want = dz.sum(0) + keep * db0
    tol = (m + 2) * 2.0 ** -23 * np.abs(dz).sum(0) + 2.0 ** -17 * np.abs(dz).sum(0) * (pre is not None)
    check(db, want, tol + last * np.abs(want) + 2.0 ** -23 * np.abs(keep * db0) + 1e-30, "dbias")


@pytest.mark.parametrize("pitch,offset", [(8, 0), (1, 0), (0, 1), (3, 5), (64, 8)])
@pytest.mark.parametrize("shape", [(1, 256, 128), (7, 96, 264), (130, 200, 136), (300, 264, 520)])
def test_pitches_and_offsets(shape, pitch, offset):
    """Views: any row pitch, any 2-byte address; what lies between the rows is not touched."""
    m, k, n = shape
    kw = dict(pitch=pitch, offset=offset)
    x, w = normal((m, k), 1.0, 1, **kw), normal((n, k), 0.1, 2, **kw)
    res, y, pre = normal((m, n), 1.0, 3, **kw), empty((m, n), **kw), empty((m, n), **kw)
    bias = normal((1, n), 1.0, 4, offset=offset)[0]
    za.zero_linear_forward(x, w, y, bias=bias, act=3, residual=res, pre=pre)
    y2, pre2 = empty((m, n)), empty((m, n))
    za.zero_linear_forward(x.contiguous(), w.contiguous(), y2, bias=bias.clone(), act=3,
                           residual=res.contiguous(), pre=pre2)
    assert torch.equal(y, y2) and torch.equal(pre, pre2)
    dy = normal((m, n), 1.0, 5, **kw)
    out = [empty((m, k), **kw), empty((n, k), F32, **kw), empty((1, n), F32, offset=offset)[0]]
    out2 = [empty((m, k)), empty((n, k), F32), empty((1, n), F32)[0]]
    za.zero_linear_backward(dy, x, w, dx=out[0], dw=out[1], dbias=out[2], act=2, pre=pre)
    za.zero_linear_backward(dy.contiguous(), x.contiguous(), w.contiguous(), dx=out2[0], dw=out2[1],
                            dbias=out2[2], act=2, pre=pre2)
    for a, b in zip(out, out2):
        assert torch.equal(a, b)
    for t in (y, pre, *out):
        if t.dim() == 2 and pitch:
            whole = t.as_strided((t.shape[0] - 1, pitch), (t.stride(0), 1), t.storage_offset() + t.shape[1])
            assert bool((whole == 7.0).all())
        assert bool((t.as_strided((offset,), (1,), 0) == 7.0).all())


@pytest.mark.parametrize("shape", [(17, 2048, 96), (64, 4096, 256), (100, 3000, 1031), (128, 2048, 130),
                                   (128, 4096, 4096), (250, 2304, 761), (256, 2304, 768),
                                   (300, 4096, 1024), (513, 1900, 200)])
def test_few_tiles_and_long_sums(shape):
    """Products whose reduction is shared out: forward, and with the widths changed over the
    gradient of x times a slope."""
    m, k, n = shape
    test_forward(shape, "gelu")
    dy, w, pre = normal((m, k), 1.0, 1), normal((k, n), 1.0 / math.sqrt(k), 2), normal((m, n), 1.0, 3)
    dx = empty((m, n))
    za.zero_linear_backward(dy, None, w, dx=dx, act_in=o.ACTS["relu"], pre_in=pre)
    want = (host(dy) @ host(w)) * (host(pre) > 0)
    tol = product_error(dy, w, k) + 2.0 ** -8 * np.abs(want) + 1e-30
    check(dx, want, tol, "dx")


@pytest.mark.parametrize("n", [17, 23, 39, 40, 41, 65, 71, 103, 135, 161, 255, 259, 263, 519])
@pytest.mark.parametrize("gap,offset", [(1, 0), (2, 3), (8, 5)])
def test_rows_at_any_address(n, gap, offset):
    """Outputs and what is added to them, in place too, at every distance from 16-byte
    boundaries, a warp's columns ending anywhere: the aligned matrices' results, and what
    lies around the rows untouched."""
    m, k = 165, 72
    kw = dict(pitch=n + gap, offset=offset)

    def moved(t):
        out = torch.full((t.shape[0] * kw["pitch"] + 64,), 7.0, dtype=t.dtype, device="cuda")
        view = out.as_strided(t.shape, (kw["pitch"], 1), offset)
        view.copy_(t)
        return out, view

    def untouched(out, view):
        keep = torch.ones(out.shape, dtype=torch.bool, device="cuda")
        keep.as_strided(view.shape, view.stride(), offset).fill_(False)
        return bool((out[keep] == 7.0).all())

    x, w = normal((m, k), 1.0, 1), normal((n, k), 0.1, 2)
    even = dict(pitch=-n % 8)
    y, pre, bias = normal((m, n), 1.0, 3, **even), empty((m, n), **even), normal((1, n), 1.0, 5)[0]
    (ybuf, yv), (pbuf, pv) = moved(y), moved(pre)
    za.zero_linear_forward(x, w, y, bias=bias, act=2, residual=y, pre=pre)
    za.zero_linear_forward(x, w, yv, bias=bias, act=2, residual=yv, pre=pv)
    assert torch.equal(yv, y) and torch.equal(pv, pre)
    assert untouched(ybuf, yv) and untouched(pbuf, pv)
    # n as the width in: dx times a slope, dw added to what is there
    dy, wt, xt = normal((m, k), 1.0, 6), normal((k, n), 0.1, 7, **even), normal((m, n), 1.0, 8, **even)
    for dtype in (BF, F32):
        dx, dw = empty((m, n), **even), empty((k, n), dtype, **even)
        dw.copy_(normal((k, n), 1.0, 9))
        (dxbuf, dxv), (dwbuf, dwv), (_, before) = moved(dx), moved(dw), moved(xt)
        za.zero_linear_backward(dy, xt, wt, dx=dx, dw=dw, act_in=2, pre_in=xt, accumulate=True)
        za.zero_linear_backward(dy, xt, wt, dx=dxv, dw=dwv, act_in=2, pre_in=before, accumulate=True)
        assert torch.equal(dxv, dx) and torch.equal(dwv, dw), dtype
        assert untouched(dxbuf, dxv) and untouched(dwbuf, dwv)


@pytest.mark.parametrize("shape", [(3, 128, 64), (200, 128, 264), (260, 72, 131)])
def test_a_bias_at_any_address(shape):
    """The bias alone is off a 16-byte boundary (a vector among others in a flat one); the
    workspace holds its copy and no more."""
    m, k, n = shape
    x, w, res = normal((m, k), 1.0, 1), normal((n, k), 0.1, 2), normal((m, n), 1.0, 3)
    moved = normal((1, n), 1.0, 4, offset=3)[0]
    bias = moved.clone()
    assert moved.data_ptr() % 16 == 6 and bias.data_ptr() % 16 == 0
    y, pre, y2, pre2 = (empty((m, n)) for _ in range(4))
    za.zero_linear_forward(x, w, y, bias=bias, act=2, residual=res, pre=pre)
    need = za.zero_linear_workspace(m, k, n)
    ws = torch.full((need + 256,), 77, dtype=torch.uint8, device="cuda")
    za.zero_linear_forward(x, w, y2, bias=moved, act=2, residual=res, pre=pre2, workspace=ws[:need])
    assert torch.equal(y, y2) and torch.equal(pre, pre2)
    assert bool((ws[need:] == 77).all())


def test_each_output_alone():
    m, k, n = 70, 130, 90
    x, w, dy, pre = (normal(s, 1.0, i) for i, s in enumerate([(m, k), (n, k), (m, n), (m, n)]))
    dx, dw, db = empty((m, k)), empty((n, k)), empty((1, n))[0]
    za.zero_linear_backward(dy, x, w, dx=dx, dw=dw, dbias=db, act=2, pre=pre)
    for name, full, kw in (("dx", dx, dict(x=None, w=w)), ("dw", dw, dict(x=x, w=None)),
                           ("dbias", db, dict(x=None, w=None))):
        alone = torch.empty_like(full)
        za.zero_linear_backward(dy, kw["x"], kw["w"], act=2, pre=pre, **{name: alone})
        assert torch.equal(alone, full), name
    za.zero_linear_backward(dy, None, None, act=2, pre=pre)      # nothing wanted


def test_no_rows():
    x, w, y = empty((0, 64)), normal((32, 64), 1.0, 1), empty((0, 32))
    za.zero_linear_forward(x, w, y)
    dw, db = empty((32, 64), F32), empty((1, 32), F32)[0]
    za.zero_linear_backward(y, x, w, dx=empty((0, 64)), dw=dw, dbias=db, accumulate=True)
    assert bool((dw == 7.0).all()) and bool((db == 7.0).all())
    za.zero_linear_backward(y, x, w, dx=empty((0, 64)), dw=dw, dbias=db)
    assert not dw.any() and not db.any()


def test_residual_in_place_and_side_by_side():
    m, d = 200, 128
    qkv = normal((m, 3 * d), 1.0, 1)
    w, before = normal((d, d), 0.1, 2), qkv.clone()
    za.zero_linear_forward(qkv[:, :d], w, qkv[:, d:2 * d], residual=qkv[:, d:2 * d])
    want = host(before[:, :d]) @ host(w).T + host(before[:, d:2 * d])
    assert np.abs(host(qkv[:, d:2 * d]) - want).max() <= 2.0 ** -7 * np.abs(want).max()
    assert torch.equal(qkv[:, :d], before[:, :d]) and torch.equal(qkv[:, 2 * d:], before[:, 2 * d:])
    with pytest.raises(za.ZeroError):
        za.zero_linear_forward(qkv[:, :d], w, qkv[:, d // 2:d // 2 + d])


@pytest.mark.parametrize("shape", [(1, 512, 256), (100, 192, 320), (300, 256, 512)])
def test_infinities_and_nan_stay_in_their_row(shape):
    """A row of x that is not finite reaches its own row of y and of dx, and no other; padding
    that the kernels read past an edge never does."""
    m, k, n = shape
    x, w = normal((m, k), 1.0, 1), normal((n, k), 0.1, 2)
    y0, y = empty((m, n)), empty((m, n))
    za.zero_linear_forward(x, w, y0, act=2)
    for bad in (float("nan"), float("inf")):
        x2 = x.clone()
        x2[m // 2, k - 1] = bad
        za.zero_linear_forward(x2, w, y, act=2)
        rows = torch.ones(m, dtype=torch.bool, device="cuda")
        rows[m // 2] = False
        assert torch.equal(y[rows], y0[rows])
        if math.isnan(bad):
            assert bool(y[m // 2].isnan().all())
        else:
            # gelu of +inf is inf, of -inf 0
            want = torch.where(w[:, k - 1] > 0, float("inf"), 0.0).to(BF)
            assert torch.equal(y[m // 2], want)


def test_activations_at_extremes():
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, 60.0, -60.0, 150.0, -150.0, 1e20, -1e20, 3e38, -3e38,
                      float("inf"), float("-inf"), float("nan")], device="cuda").to(BF)
    for name, act in o.ACTS.items():
        if act == 0:
            continue
        dx = empty((1, len(z)))
        # act_in's slope at z, times 1: a map of one feature
        za.zero_linear_backward(torch.ones(1, 1, dtype=BF, device="cuda"), None,
                                torch.ones(1, len(z), dtype=BF, device="cuda"), dx=dx, act_in=act, pre_in=z[None])
        got = host(dx)[0]
        want = o.slope(np.clip(host(z), -200, 200), name)
        assert np.isnan(got[-1]) or name == "relu"
        assert (np.abs(got[:-1] - want[:-1]) <= 2.0 ** -8 * np.abs(want[:-1]) + 2.0 ** -17).all(), (name, got)


@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
def test_gradient_against_differences(act):
    """<gradient, direction> against central differences of sum(dy * act(x w^T + b)) in 64 bits,
    along random directions of x, w and b together."""
    m, k, n = 96, 80, 72
    x, w, b, dy = normal((m, k), 1.0, 1), normal((n, k), 0.2, 2), normal((1, n), 0.5, 3)[0], normal((m, n), 1.0, 4)
    y, pre = empty((m, n)), empty((m, n))
    za.zero_linear_forward(x, w, y, bias=b, act=o.ACTS[act], pre=pre)
    dx, dw, db = empty((m, k)), empty((n, k), F32), empty((1, n), F32)[0]
    za.zero_linear_backward(dy, x, w, dx=dx, dw=dw, dbias=db, act=o.ACTS[act], pre=pre)
    hx, hw, hb, hy = host(x), host(w), host(b), host(dy)
    rng = np.random.default_rng(0)
    for _ in range(4):
        ux, uw, ub = rng.normal(size=hx.shape), rng.normal(size=hw.shape), rng.normal(size=hb.shape)

        def loss(e):
            return (hy * o.act((hx + e * ux) @ (hw + e * uw).T + hb + e * ub, act)).sum()

        h = 1e-5
        want = (loss(h) - loss(-h)) / (2 * h)
        parts = [(host(dx), ux), (host(dw), uw), (host(db), ub)]
        got = sum((g * u).sum() for g, u in parts)
        # bf16 roundings of pre, dz and dx: each good to 2^-8 of its element, independent
        size = math.sqrt(sum(((g * u) ** 2).sum() for g, u in parts))
        assert abs(got - want) <= 6 * 2.0 ** -7 * size


def test_same_bits_every_time_on_any_stream():
    m, k, n = 300, 520, 264
    x, w, dy, pre = (normal(s, 1.0, i) for i, s in enumerate([(m, k), (n, k), (m, n), (m, n)]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for stream in (None, None, side, side.cuda_stream):
        y, dx, dw, db = empty((m, n)), empty((m, k)), empty((n, k), F32), empty((1, n), F32)[0]
        side.wait_stream(torch.cuda.current_stream())
        za.zero_linear_forward(x, w, y, act=2, stream=stream)
        za.zero_linear_backward(dy, x, w, dx=dx, dw=dw, dbias=db, act=3, pre=pre, stream=stream)
        torch.cuda.synchronize()
        got.append((y, dx, dw, db))
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))
    assert za.device_status() == za.ZERO_OK


def test_in_a_graph():
    m, k, n = 128, 256, 512
    x, w, dy, pre = (normal(s, 1.0, i) for i, s in enumerate([(m, k), (n, k), (m, n), (m, n)]))
    y, dx, dw = empty((m, n)), empty((m, k)), empty((n, k))
    ws = torch.empty(za.zero_linear_workspace(m, k, n, True), dtype=torch.uint8, device="cuda")

    def both():
        za.zero_linear_forward(x, w, y, act=2, workspace=ws)
        za.zero_linear_backward(dy, x, w, dx=dx, dw=dw, act=3, pre=pre, workspace=ws)

    both()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, dx, dw)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for t in (y, dx, dw):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (y, dx, dw)))


@pytest.mark.parametrize("pitch", [2_000_000, 4_000_001])
def test_offsets_past_32_bits(pitch):
    """Rows whose element offset passes 2^31, or 2^32: the last rows of a 2.2e9-element x and
    y, and of 4.4e9 with rows on odd addresses."""
    m, k, n = 1100, 64, 64
    big = torch.empty((m - 1) * pitch + k, dtype=BF, device="cuda")
    x = big.as_strided((m, k), (pitch, 1))
    x.copy_(normal((m, k), 1.0, 1))
    w = normal((n, k), 0.1, 2)
    y2 = empty((m, n))
    za.zero_linear_forward(x.contiguous(), w, y2)
    out = torch.empty((m - 1) * pitch + n, dtype=BF, device="cuda").as_strided((m, n), (pitch, 1))
    za.zero_linear_forward(x, w, out)
    assert torch.equal(out, y2)


@pytest.mark.parametrize("rows", [1, 700, 4096, 16384])
def test_fp32_gradients_keep_their_precision(rows):
    """The tensor cores cut sums off, by 1e-9 of a sum a step: fp32 gradients of many rows
    are within 1e-6 of the exact ones in the 2-norm (one chain of 16,384 steps: 1.6e-5)."""
    x, dy = normal((rows, 256), 1.0, 1), normal((rows, 384), 1.0, 2)
    dw, db = empty((384, 256), F32), empty((1, 384), F32)[0]
    za.zero_linear_backward(dy, x, None, dw=dw, dbias=db)
    want = host(dy).T @ host(x)
    assert np.linalg.norm(host(dw) - want) <= 1e-6 * np.linalg.norm(want)
    want = host(dy).sum(0)
    assert np.linalg.norm(host(db) - want) <= 1e-6 * np.linalg.norm(want)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("m", [4, 200])
def test_order_among_streams(m, captured):
    """Calls begin while their stream's last kernel ends: what another stream wrote before an
    event is read, and what is overwritten after one has been read, run or captured."""
    k, n = 512, 768
    x, w, dy = normal((m, k), 1.0, 1), normal((n, k), 0.1, 2), normal((m, n), 1.0, 3)
    y, dx, dw, db = empty((m, n)), empty((m, k)), empty((n, k)), empty((1, n))[0]
    want = [torch.empty_like(t) for t in (y, dx, dw, db)]
    za.zero_linear_forward(x, w, want[0])
    za.zero_linear_backward(dy, x, w, dx=want[1], dw=want[2], dbias=want[3], act=2, pre=want[0])
    inputs, late = (x, w, dy), [torch.zeros_like(t) for t in (x, w, dy)]
    copies = [torch.empty_like(t) for t in want]
    tiny = torch.zeros(1, device="cuda")
    a, b = torch.cuda.Stream(), torch.cuda.Stream()

    def work(a, b):
        b.wait_stream(a)
        with torch.cuda.stream(b):
            torch.cuda._sleep(2_000_000)
            for t, s in zip(late, inputs):
                t.copy_(s)
        with torch.cuda.stream(a):
            tiny.add_(1.0)               # a kernel right before the call, beside the event
            a.wait_stream(b)
            za.zero_linear_forward(late[0], late[1], y)
            za.zero_linear_backward(late[2], late[0], late[1], dx=dx, dw=dw, dbias=db, act=2, pre=y)
        b.wait_stream(a)
        with torch.cuda.stream(b):
            for t, s in zip(copies, (y, dx, dw, db)):
                t.copy_(s)
            for t in (*late, y, dx, dw, db):
                t.zero_()
        a.wait_stream(b)

    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=a):
            work(a, b)
        for _ in range(3):
            graph.replay()
    else:
        for _ in range(3):
            work(a, b)
    torch.cuda.synchronize()
    for got, t in zip(copies, want):
        assert torch.equal(got, t)


def test_a_wait_that_runs_out_is_reported():
    """With no tile loaded every wait of the product gives up after about a second, nothing
    is written, the status says so, and the next call is as if nothing had been."""
    x, w, y = normal((200, 256), 1.0, 1), normal((320, 256), 0.1, 2), empty((200, 320))
    dx, dw = empty((200, 256)), empty((320, 256), F32)
    dy = normal((200, 320), 1.0, 3)
    assert za.device_status() == za.ZERO_OK
    was = za.test_withhold_copies(True)
    try:
        za.zero_linear_forward(x, w, y)
        torch.cuda.synchronize()
        assert za.device_status() == -15
        assert bool((y == 7.0).all())
        za.zero_linear_backward(dy, x, w, dx=dx, dw=dw)
        torch.cuda.synchronize()
        assert za.device_status() == -15
        assert bool((dx == 7.0).all()) and bool((dw == 7.0).all())
        x2, w2, y2 = normal((128, 2048), 1.0, 4), normal((256, 2048), 0.1, 5), empty((128, 256))
        za.zero_linear_forward(x2, w2, y2)    # a reduction shared out in a cluster
        torch.cuda.synchronize()
        assert za.device_status() == -15
        assert bool((y2 == 7.0).all())
    finally:
        za.test_withhold_copies(was)
    assert za.device_status() == za.ZERO_OK
    za.zero_linear_forward(x, w, y)
    want = host(x) @ host(w).T
    assert np.abs(host(y) - want).max() <= 2.0 ** -7 * np.abs(want).max()
    assert za.device_status() == za.ZERO_OK


def test_few_rows_of_the_greatest_width():
    """in = 2^31 - 2, the largest taken: the columns past the last whole round are counted
    without overflow.  Zeros but for ones at both ends and in between, so sums are exact."""
    k = 2 ** 31 - 2
    x = torch.zeros(2, k + 2, dtype=BF, device="cuda")[:, :k]
    w = torch.zeros(3, k + 2, dtype=BF, device="cuda")[:, :k]
    at = torch.tensor([0, 5, 1023, 2 ** 30, k - 2000, k - 1025, k - 1024, k - 9, k - 2, k - 1], device="cuda")
    x[0, at], x[1, at[::2]] = 1.0, 2.0
    w[0, at], w[1, at[-1]], w[2, at[1:]] = 1.0, 3.0, 1.0
    y = empty((2, 3))
    za.zero_linear_forward(x, w, y)
    assert y.tolist() == [[10.0, 3.0, 9.0], [10.0, 0.0, 8.0]]


@pytest.mark.parametrize("handle", [False, True])
def test_a_call_on_another_stream_leaves_freed_memory_alone(handle):
    """Memory that the current stream has freed but not yet done with is not the workspace of
    a call on another stream, which may run long before."""
    m, k, n = 300, 520, 264
    x, w, dy, pre = (normal(s, 1.0, i) for i, s in enumerate([(m, k), (n, k), (m, n), (m, n)]))
    dx, dw = empty((m, k)), empty((n, k), F32)
    need = za.zero_linear_workspace(m, k, n, True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # of the sizes that a workspace may have, in one block or in parts of one
    temporaries = [torch.full((size,), 77, dtype=torch.uint8, device="cuda") for size in (need, need, 20 << 20)]
    seen = [torch.empty_like(t) for t in temporaries]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    for t, s in zip(temporaries, seen):
        s.copy_(t)
    del temporaries, t
    for _ in range(4):
        za.zero_linear_backward(dy, x, w, dx=dx, dw=dw, act=3, pre=pre,
                                stream=side.cuda_stream if handle else side)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(bool((s == 77).all()) for s in seen)


@pytest.mark.parametrize("shape", o.SHARED_ROUNDS)
@pytest.mark.parametrize("act,act_in,dtype,add", [("none", "silu", F32, True), ("silu", "none", BF, False)])
def test_shared_rounds_of_dx_and_dw(shape, act, act_in, dtype, add):
    """dw's tiles go round several times among the units that dx's last round leaves idle."""
    test_backward(shape, act, act_in, dtype, add)


@pytest.mark.parametrize("shape", [(130, 200, 136), (300, 775, 1031), (777, 768, 2304), (1003, 71, 2311)])
@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
def test_backward_against_the_rounded_dz(shape, act):
    """dx and dw are products of dz = bf16(dy act'(pre)): held to an fp32 product's error of
    those, which is far below what the rounding itself may do.  The slope is good to 2^-17, so
    an element of dz that lies that near to a rounding boundary may be its other neighbour."""
    m, k, n = shape
    x, w, dy = normal((m, k), 1.0, 1), normal((n, k), 1.0 / math.sqrt(k), 2), normal((m, n), 1.0, 3)
    pre = normal((m, n), 1.0, 4)
    dx, dw = empty((m, k)), empty((n, k), F32)
    za.zero_linear_backward(dy, x, w, dx=dx, dw=dw, act=o.ACTS[act], pre=pre)
    exact = host(dy) * o.slope(host(pre), act)
    # what 2^-17 of a slope near 0 is to dz is not relative to dz itself
    near = 2.0 ** -17 * (np.abs(exact) + np.abs(host(dy)))
    low, dz, high = (o.round_bf16((exact + d).astype(np.float32)).astype(np.float64) for d in (-near, 0.0, near))
    edz = torch.from_numpy(high - low).cuda()
    dz = torch.from_numpy(dz).cuda()
    want = host(dz @ w.double())
    tol = product_error(dz, w, n) + host(edz @ w.double().abs()) + 2.0 ** -8 * np.abs(want) + 1e-30
    check(dx, want, tol, "dx")
    want = host(dz.t() @ x.double())
    check(dw, want, product_error(dz.t(), x, m) + host(edz.t() @ x.double().abs()) + 1e-30, "dw")


@pytest.mark.parametrize("m", [1, 16, 40, 300])
@pytest.mark.parametrize("d", [256, 515, 1024])
def test_one_calls_output_is_the_nexts_input(m, d):
    """Layers in a row on one stream, each adding to its input in place and the next reading
    that, called without a pause (a kernel begins while the one before ends): the bits of the
    same calls with the GPU waited for after each."""
    ws = [normal((d, d), 0.3 / math.sqrt(d), i) for i in range(4)]
    x0, space = normal((m, d), 1.0, 9), torch.empty(za.zero_linear_workspace(m, d, d, True) + 16, dtype=torch.uint8, device="cuda")
    dy0 = normal((m, d), 1.0, 10)

    def layers(wait):
        x, mid, dy, dw = x0.clone(), empty((m, d)), dy0.clone(), empty((d, d), F32)
        for _ in range(10):
            for w in ws:
                za.zero_linear_forward(x, w, mid, act=3, workspace=space)
                wait()
                za.zero_linear_forward(mid, w, x, residual=x, workspace=space)
                wait()
                za.zero_linear_backward(dy, x, w, dx=mid, dw=dw, act=3, pre=x, workspace=space, accumulate=True)
                wait()
                za.zero_linear_forward(mid, w, dy, residual=dy, workspace=space)
                wait()
                x.mul_(0.7)
                dy.mul_(0.7)
        torch.cuda.synchronize()
        return x, dy, dw

    want = layers(torch.cuda.synchronize)
    assert all(bool(t.isfinite().all()) for t in want)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(layers(lambda: None), want))
