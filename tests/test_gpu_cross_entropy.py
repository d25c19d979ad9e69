"""Softmax cross entropy of a linear map and its gradients on the GPU against 64 bits."""
import math

import pytest
import torch

import model_oracle as o
import zero_partitioned_mixed_adam_gb300 as za

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64

# rows, width, vocabulary: ones; around tiles of 32 to 256 columns and 128 rows; odd; longer
SHAPES = [(1, 1, 1), (1, 64, 2), (2, 8, 33), (3, 33, 7), (16, 8, 100), (37, 256, 515), (64, 130, 31),
          (127, 64, 256), (128, 128, 255), (129, 72, 257), (200, 775, 1031), (257, 320, 4099),
          (300, 64, 50257), (700, 2048, 1000), (1500, 24, 3001)]


def matrix(rows, cols, sigma, seed, pitch=0, offset=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    flat = torch.empty(offset + rows * (cols + pitch), device="cuda").normal_(0, sigma, generator=gen).to(BF)
    return flat[offset:].view(rows, cols + pitch)[:, :cols]


def blank(rows, cols, dtype=BF, pitch=0, offset=0):
    flat = torch.full((offset + rows * (cols + pitch),), 7.0, dtype=dtype, device="cuda")
    return flat[offset:].view(rows, cols + pitch)[:, :cols]


def targets_of(rows, vocab, seed, ignored=0.0, ignore=-100, dtype=torch.int64):
    gen = torch.Generator("cuda").manual_seed(seed)
    t = torch.randint(0, vocab, (rows,), device="cuda", generator=gen)
    return torch.where(torch.rand(rows, device="cuda", generator=gen) < ignored, ignore, t).to(dtype)


def tolerances(x, w, ref):
    """Bounds (losses, dx, dw before their own rounding) on what the kernels' arithmetic may
    put in.

    z: sums of 16 products or more at a time, each of the width/16 + 2 additions good to 2^-22
    of the sum of magnitudes so far, and the reference's alike.  The sum of exponentials: each
    within its argument's error, 2^-19 of argument times 2^-24 and 2 ulp (arguments up to 45),
    100 additions of 2^-24: 2^-17 in all.  dz: the sum's error, 2^-8 for an exponential's rounding to
    bf16, and 2^-8 more: dz's own rounding, or the target's, which the row's factor takes over.  What
    is below exp(-87) of the reference's is nothing.  dw of more than 2^25 values: 2^-8 for x times the
    factor, in bf16, and there the target's dz is exact.  Products: as z."""
    losses, _, _, _, dz, z, c = ref
    keep = (c != 0)[:, None]
    ax, aw = torch.where(keep, x.to(F64).abs(), 0.0), w.to(F64).abs()
    width, vocab, rows = x.shape[1], w.shape[0], x.shape[0]
    ez = 2 * ((width / 16 + 2) * 2.0 ** -22 * (ax @ aw.t())).amax(1)
    rel = 2 * ez + 2.0 ** -17
    tol_loss = rel * -torch.expm1(-losses) + 2.0 ** -22 * losses.abs() + 1e-12 + ez * (losses > 30)
    ddz = dz.abs() * (torch.where(dz * c[:, None] > 0, 2.0 ** -7, 2.0 ** -8) + rel[:, None]) * 1.01
    ddz = ddz + math.exp(-87) * c[:, None].abs()
    fdw = 2.0 ** -8 if rows * vocab > 2 ** 25 else 0.0
    adz = dz.abs() + ddz
    tol_dx = ddz @ aw + (vocab / 16 + 2) * 2.0 ** -22 * (adz @ aw)
    tol_dw = (ddz + fdw * adz).t() @ ax + (rows / 16 + 2) * 2.0 ** -22 * (adz.t() @ ax)
    return tol_loss, tol_dx, tol_dw


def near(got, want, tol, what):
    assert torch.isfinite(got).all(), what
    bad = (got.to(F64) - want).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), float(((got.to(F64) - want).abs() - tol).max()))


def check(x, w, t, *, scale=None, dtype=BF, add=False, dx=None, dw=None, ignore=-100, **kw):
    rows, vocab = x.shape[0], w.shape[0]
    losses, total = torch.full((rows,), 7.0, device="cuda"), torch.full((1,), 7.0, device="cuda")
    dx = blank(*x.shape) if dx is None else dx
    dw = blank(*w.shape, dtype=dtype) if dw is None else dw
    before = dw.to(F64)
    za.zero_linear_cross_entropy(x, w, t, losses, total, dx=dx, dw=dw, scale=scale, accumulate=add,
                                 ignore_index=ignore, **kw)
    ref = o.cross_entropy(x, w, t, ignore, scale)
    tol_loss, tol_dx, tol_dw = tolerances(x, w, ref)
    near(losses, ref[0], tol_loss, "losses")
    near(total, ref[1], (tol_loss * ref[6].abs()).sum() + 2.0 ** -22 * (ref[6] * ref[0]).abs().sum(), "total")
    near(dx, ref[2], tol_dx + 2.0 ** -8 * ref[2].abs() + 1e-30, "dx")
    want = ref[3] + before if add else ref[3]
    half = 2.0 ** -8 if dw.dtype == BF else 2.0 ** -23
    near(dw, want, tol_dw + half * (want.abs() + tol_dw) + 1e-30, "dw")
    assert za.device_status() == za.ZERO_OK
    check_alone(x, w, t, ref, scale=scale, ignore_index=ignore)
    return losses, total, dx, dw, ref


def check_alone(x, w, t, ref, **kw):
    """The loss without gradients, which other kernels compute: each exponential once less the
    largest logit and once more less the target's, so twice the error of the sum."""
    losses, total = torch.full(t.shape, 7.0, device="cuda"), torch.full((1,), 7.0, device="cuda")
    za.zero_linear_cross_entropy(x, w, t, losses, total, **kw)
    tol = tolerances(x, w, ref)[0] + 2.0 ** -17 * -torch.expm1(-ref[0])
    near(losses, ref[0], tol, "losses alone")
    near(total, ref[1], (tol * ref[6].abs()).sum() + 2.0 ** -22 * (ref[6] * ref[0]).abs().sum(), "total alone")


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("ignored,ids", [(0.0, torch.int64), (0.4, torch.int32)])
def test_loss_and_gradients(shape, ignored, ids):
    m, k, v = shape
    t = targets_of(m, v, 3, ignored, dtype=ids)
    if (t == -100).all():
        t[0] = 0
    check(matrix(m, k, 1.0, 1), matrix(v, k, 1.5 / math.sqrt(k), 2), t)


@pytest.mark.parametrize("shape", SHAPES[::3])
@pytest.mark.parametrize("dtype,add", [(BF, True), (F32, False), (F32, True)])
def test_scales_types_and_accumulation(shape, dtype, add):
    m, k, v = shape
    scale = torch.linspace(-1.0, 2.0, m, device="cuda")
    t = targets_of(m, v, 4, 0.2)
    dw = matrix(v, k, 0.1, 5).to(dtype)
    check(matrix(m, k, 1.0, 1), matrix(v, k, 1.0 / math.sqrt(k), 2), t, scale=scale, add=add, dw=dw, dtype=dtype)


@pytest.mark.parametrize("shape", [(37, 256, 515), (130, 75, 301), (64, 64, 64)])
@pytest.mark.parametrize("pitch,offset", [(0, 1), (1, 0), (8, 8), (3, 5)])
def test_layouts(shape, pitch, offset):
    m, k, v = shape
    dx, dw = blank(m, k, pitch=pitch, offset=offset), blank(v, k, pitch=pitch, offset=offset)
    around = [(b._base, b) for b in (dx, dw)]
    check(matrix(m, k, 1.0, 1, pitch, offset), matrix(v, k, 0.1, 2, pitch, offset), targets_of(m, v, 3), dx=dx, dw=dw)
    for flat, view in around:      # what lies between the rows and before them is as it was
        view.fill_(7.0)
        assert (flat == 7.0).all()


def test_parts_alone():
    """Each output alone is what it is with the others."""
    m, k, v = 150, 96, 700
    x, w, t = matrix(m, k, 1.0, 1), matrix(v, k, 0.2, 2), targets_of(m, v, 3, 0.1)
    losses, total, dx, dw, _ = check(x, w, t)
    for name, want in (("dx", dx), ("dw", dw)):
        got = torch.full_like(want, 7.0)
        za.zero_linear_cross_entropy(x, w, t, **{name: got})
        assert torch.equal(got, want), name
    alone = [torch.full_like(losses, 7.0), torch.full_like(total, 7.0)]
    za.zero_linear_cross_entropy(x, w, t, *alone)     # no gradients
    for name, want in (("losses", alone[0]), ("total", alone[1])):
        got = torch.full_like(want, 7.0)
        za.zero_linear_cross_entropy(x, w, t, **{name: got})
        assert torch.equal(got, want), name


@pytest.mark.parametrize("rows,k,v", [(3, 64, 1000), (140, 64, 1000), (40, 75, 333), (300, 256, 4099)])
def test_far_targets(rows, k, v):
    """Targets far below the largest logit (losses of 40 to 400: another reference is taken, by the
    rows' own blocks up to 2^28 products and by a second run of the product beyond), far above
    all others, and both among ordinary rows."""
    x, w = matrix(rows, k, 1.0, 1), matrix(v, k, 1.0, 2)
    t = targets_of(rows, v, 3)
    z = x.float() @ w.float().t()
    t[0] = z[0].argmin()
    t[1] = z[1].argmax()
    x[0] *= 8.0
    x[1] *= 8.0
    losses, *_ = check(x, w, t)
    assert losses[0] > 100 and losses[1] < 1e-3
    check((x * 4.0), w, t)                       # most rows


@pytest.mark.parametrize("v", [2, 515, 50257, 131072])
def test_targets_below_a_plateau(v):
    """All other logits alike and 30 to 100 above the target's: the exponentials' sum less the target's
    passes fp32's range from a loss of 88.7 on, whatever its largest term is."""
    depth = torch.arange(30.0, 100.5, 0.5, device="cuda")
    x, w = blank(len(depth), 8), blank(v, 8)
    x.zero_(), w.zero_()
    x[:, 0], w[:, 0] = depth.to(BF), 1.0
    at = min(7, v - 1)
    w[at] = 0.0
    t = torch.full((len(depth),), at, device="cuda")
    losses, *_ = check(x, w, t)
    assert losses.max() > 99
    check(x, w, t, scale=torch.linspace(-1.0, 2.0, len(depth), device="cuda"), dtype=F32)


@pytest.mark.parametrize("rows,k,v", [(5, 64, 7), (700, 64, 40), (1300, 75, 3), (601, 16, 64), (601, 16, 65)])
def test_far_targets_of_few_columns(rows, k, v):
    """Rows of few columns, a warp's or a block's, most of them with another reference; some ignored."""
    x, w = matrix(rows, k, 1.0, 1), matrix(v, k, 1.0, 2)
    t = targets_of(rows, v, 3, 0.2)
    t[0] = 0
    check(x, w, t)
    losses, *_ = check(x * 16.0, w, t)
    assert (losses > 50).any()


@pytest.mark.parametrize("rows,k,v", [(1, 64, 50257), (2, 2048, 4099), (7, 775, 9001), (130, 520, 5003)])
def test_few_rows_of_many_columns(rows, k, v):
    """More weights than one block reads again for a row: another reference is a second run of the
    product for few rows too, and dz is made in place."""
    assert rows * v <= 2 ** 25 and k * v > 2 ** 21
    x, w = matrix(rows, k, 1.0, 1), matrix(v, k, 2.0 / math.sqrt(k), 2)
    t = targets_of(rows, v, 3)
    check(x, w, t)
    x[0] *= 32.0
    t[0] = (x[0].float() @ w.float().t()).argmin()
    if rows > 2:
        t[1] = -100
        x[1] = float("nan")
    losses, *_ = check(x, w, t)
    assert losses[0] > 60


def test_certain_rows():
    """A model that is sure of its target: 1 - p_t as small as 1e-9 comes out to its last bits."""
    k, v = 32, 300
    w = matrix(v, k, 0.5, 2)
    t = targets_of(64, v, 3)
    x = (torch.linspace(1.0, 6.0, 64, device="cuda")[:, None] * w[t].float()).to(BF)
    losses, _, dx, _, ref = check(x, w, t)
    small = ref[0] < 1e-5
    assert small.any() and ((losses - ref[0]).abs() <= 1e-3 * ref[0] + 1e-12)[small].all()


def test_ignored_rows_may_hold_anything():
    m, k, v = 100, 72, 333
    x, w, t = matrix(m, k, 1.0, 1), matrix(v, k, 0.2, 2), targets_of(m, v, 3, 0.3)
    x[t == -100] = float("inf")
    x[(t == -100).nonzero()[0]] = float("nan")
    losses, _, dx, _, _ = check(x, w, t)
    assert (losses[t == -100] == 0).all() and (dx[t == -100] == 0).all()


def test_every_row_ignored():
    m, k, v = 70, 64, 100
    t = torch.full((m,), 5, device="cuda")
    x = torch.full((m, k), float("nan"), device="cuda", dtype=BF)
    losses, total, dx, dw = (torch.full(s, 7.0, device="cuda") for s in ((m,), (1,), (m, k), (v, k)))
    dx = dx.to(BF)
    w = matrix(v, k, 1.0, 2)
    za.zero_linear_cross_entropy(x, w, t, losses, total, dx=dx, dw=dw, ignore_index=5)
    assert not any(a.any() for a in (losses, total, dx, dw))
    losses.fill_(7.0), total.fill_(7.0)
    za.zero_linear_cross_entropy(x, w, t, losses, total, ignore_index=5)
    assert not losses.any() and not total.any()


@pytest.mark.parametrize("count", [0, 1, 5, 128, 129, 700, 1023, 1024])
@pytest.mark.parametrize("k,pitch", [(256, 0), (263, 5)])
def test_rows_that_count_are_done_alone(count, k, pitch):
    """Beyond 2^28 products ignored rows are left out of them: as many as there are, wherever they
    lie, whatever they hold, to the bits of a call without them."""
    m, v = 1024, 2000
    assert m * k * v > 2 ** 28
    gen = torch.Generator("cuda").manual_seed(count)
    t = targets_of(m, v, 3)
    t[torch.randperm(m, device="cuda", generator=gen)[count:]] = -100
    x, w = matrix(m, k, 1.0, 1, pitch), matrix(v, k, 0.2, 2)
    x[t == -100] = float("nan")
    if count == 0:
        out = [torch.full(s, 7.0, device="cuda") for s in ((m,), (1,), (m, k), (v, k))]
        out[2] = out[2].to(BF)
        za.zero_linear_cross_entropy(x, w, t, out[0], out[1], dx=out[2], dw=out[3])
        assert not any(a.any() for a in out)
        return
    losses, total, dx, dw, _ = check(x, w, t, dx=blank(m, k, pitch=pitch))
    assert (losses[t == -100] == 0).all() and (dx[t == -100] == 0).all()
    scale = torch.linspace(-1.0, 2.0, m, device="cuda")
    scale[t == -100] = float("inf")
    check(x, w, t, scale=torch.where(t == -100, 0.0, scale), dtype=F32, add=True, dw=matrix(v, k, 0.1, 5).float())
    again = torch.zeros(m, device="cuda")
    za.zero_linear_cross_entropy(x, w, t, again, total, dx=dx, scale=scale)
    assert torch.isfinite(total).all() and torch.isfinite(dx).all()


def test_no_rows():
    w = matrix(9, 16, 1.0, 1)
    x, t = w[:0], torch.empty(0, dtype=torch.int64, device="cuda")
    total, dw = torch.full((1,), 7.0, device="cuda"), blank(9, 16)
    za.zero_linear_cross_entropy(x, w, t, None, total, dw=dw, accumulate=True)
    assert total == 0 and (dw == 7.0).all()
    za.zero_linear_cross_entropy(x, w, t, None, total, dx=x.clone(), dw=dw)
    assert not dw.any()


@pytest.mark.parametrize("bad", [-1, 333, 2 ** 40])
def test_targets_that_are_no_column(bad):
    m, k, v = 40, 72, 333
    x, w, t = matrix(m, k, 1.0, 1), matrix(v, k, 0.2, 2), targets_of(m, v, 3)
    want = o.cross_entropy(x, w, t)[0]
    t[7] = bad
    losses, total, dx = torch.zeros(m, device="cuda"), torch.zeros(1, device="cuda"), blank(m, k)
    za.zero_linear_cross_entropy(x, w, t, losses, total, dx=dx)
    assert losses[7].isnan() and total.isnan().all() and dx[7].isnan().all()
    others = torch.arange(m, device="cuda") != 7
    assert ((losses - want).abs() < 1e-4)[others].all() and torch.isfinite(dx[others]).all()
    losses.fill_(7.0), total.fill_(7.0)
    za.zero_linear_cross_entropy(x, w, t, losses, total)
    assert losses[7].isnan() and total.isnan().all() and ((losses - want).abs() < 1e-4)[others].all()


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_rows_that_are_not_finite(value):
    m, k, v = 40, 64, 100
    x, w, t = matrix(m, k, 1.0, 1), matrix(v, k, 0.2, 2).abs(), targets_of(m, v, 3)
    x[5, 3] = value
    losses, dx = torch.zeros(m, device="cuda"), blank(m, k)
    za.zero_linear_cross_entropy(x, w, t, losses, dx=dx)
    others = torch.arange(m, device="cuda") != 5
    assert not torch.isfinite(losses[5]) and not torch.isfinite(dx[5]).any()
    assert torch.isfinite(losses[others]).all() and torch.isfinite(dx[others]).all()
    alone = torch.zeros(m, device="cuda")
    za.zero_linear_cross_entropy(x, w, t, alone)
    assert not torch.isfinite(alone[5]) and torch.isfinite(alone[others]).all()


@pytest.mark.parametrize("dtype,add", [(BF, False), (BF, True), (F32, True)])
def test_rows_in_pieces(dtype, add):
    """More rows than one piece of a GiB holds: dw is the pieces' sum, rounded once."""
    m, k, v = 4608, 32, 131072
    assert 2 * m * v > 2 ** 30
    dw = matrix(v, k, 1e-4, 5).to(dtype)
    check(matrix(m, k, 1.0, 1), matrix(v, k, 0.3, 2), targets_of(m, v, 3, 0.1), dtype=dtype, add=add, dw=dw)


# more than 2^25 values: the exponentials stay as they are, and x and dx take the rows' factors
MANY = [(1100, 40, 32003), (2100, 264, 16411), (700, 75, 50257)]


@pytest.mark.parametrize("m,k,v", MANY)
@pytest.mark.parametrize("ignored,pitch", [(0.0, 0), (0.4, 3)])
def test_many_values(m, k, v, ignored, pitch):
    t = targets_of(m, v, 3, ignored)
    x, w = matrix(m, k, 1.0, 1, pitch), matrix(v, k, 2.0 / math.sqrt(k), 2, pitch)
    x[t == -100] = float("nan")
    check(x, w, t, dx=blank(m, k, pitch=pitch), dw=blank(v, k, pitch=pitch))
    scale = torch.linspace(-1.0, 2.0, m, device="cuda")
    first = check(x, w, t, scale=scale, dtype=F32, add=True, dw=matrix(v, k, 0.1, 5).float())
    for name, at in (("dx", 2), ("dw", 3)):          # each alone, to the same bits
        got = matrix(v, k, 0.1, 5).float() if name == "dw" else torch.full_like(first[2], 7.0)
        za.zero_linear_cross_entropy(x, w, t, scale=scale, accumulate=name == "dw", **{name: got})
        assert torch.equal(got, first[at]), name


@pytest.mark.parametrize("m,k,v", MANY[::2])
def test_many_values_far_targets(m, k, v):
    """Rows that take the largest logit for their reference beside ordinary and certain ones, then
    most rows of the first kind."""
    x, w = matrix(m, k, 1.0, 1), matrix(v, k, 1.0, 2)
    t = targets_of(m, v, 3, 0.1)
    z = x.float() @ w.float().t()
    t[0], t[1] = z[0].argmin(), z[1].argmax()
    x[0] *= 16.0
    x[1] *= 16.0
    losses, *_ = check(x, w, t)
    assert losses[0] > 100 and losses[1] < 1e-3
    check(x * 8.0, w, t)


def test_many_values_that_are_not_good():
    """A target that is no column and a row that is not finite spoil their own losses and dx."""
    m, k, v = MANY[0]
    x, w, t = matrix(m, k, 1.0, 1), matrix(v, k, 0.2, 2), targets_of(m, v, 3, 0.1)
    t[4] = t[7] = t[9] = 1
    want = o.cross_entropy(x, w, t)[0]
    t[4], x[7, 3], x[9, 5] = v, float("inf"), float("nan")
    losses, total, dx, dw = torch.zeros(m, device="cuda"), torch.zeros(1, device="cuda"), blank(m, k), blank(v, k)
    za.zero_linear_cross_entropy(x, w, t, losses, total, dx=dx, dw=dw)
    others = torch.ones(m, dtype=torch.bool, device="cuda")
    others[torch.tensor([4, 7, 9], device="cuda")] = False
    assert not torch.isfinite(losses[~others]).any() and not torch.isfinite(dx[~others]).any()
    assert ((losses - want).abs() < 1e-4)[others].all() and torch.isfinite(dx[others]).all()
    assert not torch.isfinite(total).any() and not torch.isfinite(dw).any()


def test_the_same_bits_every_time():
    m, k, v = 700, 256, 3001
    x, w, t = matrix(m, k, 1.0, 1), matrix(v, k, 0.2, 2), targets_of(m, v, 3, 0.1)
    first = check(x, w, t)[:4]
    for _ in range(3):
        got = [torch.full_like(a, 7.0) for a in first]
        za.zero_linear_cross_entropy(x, w, t, got[0], got[1], dx=got[2], dw=got[3])
        assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_streams_and_graphs():
    """On another stream, with a workspace of the caller's; captured and replayed on new inputs."""
    m, k, v = 200, 128, 1031
    x, w, t = matrix(m, k, 1.0, 1), matrix(v, k, 0.2, 2), targets_of(m, v, 3, 0.1)
    want = check(x, w, t)[:4]
    need = za.zero_linear_cross_entropy_workspace(m, k, v, aligned=True)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out = [torch.full_like(a, 7.0) for a in want]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    za.zero_linear_cross_entropy(x, w, t, out[0], out[1], dx=out[2], dw=out[3], workspace=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    graph, alone = torch.cuda.CUDAGraph(), torch.zeros(m, device="cuda")
    with torch.cuda.graph(graph):
        za.zero_linear_cross_entropy(x, w, t, out[0], out[1], dx=out[2], dw=out[3])
        za.zero_linear_cross_entropy(x, w, t, alone)
    x.copy_(matrix(m, k, 4.0, 11))          # among them rows that need another reference
    w.copy_(matrix(v, k, 1.0, 12))
    t.copy_(targets_of(m, v, 13, 0.3))
    graph.replay()
    graph.replay()
    want = check(x, w, t)[:4]
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    again = torch.zeros_like(alone)
    za.zero_linear_cross_entropy(x, w, t, again)
    assert torch.equal(alone, again)


def test_withheld_copies_are_reported():
    m, k, v = 64, 64, 256
    x, w, t = matrix(m, k, 1.0, 1), matrix(v, k, 0.2, 2), targets_of(m, v, 3)
    za.test_withhold_copies(True)
    try:
        za.zero_linear_cross_entropy(x, w, t, torch.zeros(m, device="cuda"))
        assert za.device_status() != za.ZERO_OK
    finally:
        za.test_withhold_copies(False)
    check(x, w, t)


def test_gradients_against_differences():
    """dx and dw against central differences of the 64-bit loss, on a handful of entries."""
    m, k, v = 6, 16, 40
    x, w, t = matrix(m, k, 1.0, 1), matrix(v, k, 0.3, 2), targets_of(m, v, 3)
    _, _, dx, dw, _ = check(x, w, t, dtype=F32)
    step = 1e-4
    for which, grad in ((0, dx), (1, dw)):
        for i, j in ((0, 0), (3, 7), (5, 15)):
            moved = []
            for sign in (1, -1):
                pair = [x.to(F64).clone(), w.to(F64).clone()]
                pair[which][i, j] += sign * step
                moved.append(o.cross_entropy(*pair, t)[1])
            slope = (moved[0] - moved[1]) / (2 * step)
            # step^2 of the third derivative, and the gradient's own rounding
            assert (grad[i, j].to(F64) - slope).abs() <= 1e-6 + 2.0 ** -6 * grad[i].to(F64).abs().max()


@pytest.mark.parametrize("m,k,v", [(40, 64, 100), (5, 75, 33), (700, 64, 40), (300, 64, 50257), (1024, 256, 2000), (1100, 40, 32003)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_ignored_rows_beside_weights_that_are_not_finite(m, k, v, value):
    """An ignored row's loss and dx are 0 whatever is in w too; with all rows ignored so are dw and total."""
    x, w, t = matrix(m, k, 1.0, 1), matrix(v, k, 0.2, 2), targets_of(m, v, 3, 0.4)
    t[0], t[1] = -100, 1
    w[3, 5] = value
    losses, total = torch.full((m,), 7.0, device="cuda"), torch.full((1,), 7.0, device="cuda")
    dx, dw = blank(m, k), blank(v, k)
    za.zero_linear_cross_entropy(x, w, t, losses, total, dx=dx, dw=dw)
    ignored = t == -100
    assert (losses[ignored] == 0).all() and (dx[ignored] == 0).all()
    assert not torch.isfinite(dx[1]).all()     # (the weight's 0 or infinite share of a row that counts)
    t.fill_(-100)
    za.zero_linear_cross_entropy(x, w, t, losses, total, dx=dx, dw=dw)
    assert not any(a.any() for a in (losses, total, dx, dw))


@pytest.mark.parametrize("m,k,v", [(1024, 3776, 5003), (700, 4096, 4099), (300, 8200, 2051)])
def test_wide_losses_are_fp32(m, k, v):
    """The tensor cores cut off some 1e-9 of a sum at each step of the reduction, all one way, so that a
    mean of many losses does not average it out.  Chains of 768 steps leave 768e-9 of the logits,
    weighted as the loss weighs them; the loss itself is worth 2^-24 of its value, and its sum and
    logarithm 3 times that."""
    x, w, t = matrix(m, k, 1.0, 1), matrix(v, k, 0.02, 2), targets_of(m, v, 3)
    ref = o.cross_entropy(x, w, t)
    p = torch.softmax(ref[5], 1)
    tol = 768e-9 * (p * ref[5]).sum(1).abs().mean() + 4 * 2.0 ** -24 * ref[1]
    total = torch.zeros(1, device="cuda")
    za.zero_linear_cross_entropy(x, w, t, None, total)
    near(total, ref[1], tol, "alone")
    za.zero_linear_cross_entropy(x, w, t, None, total, dx=torch.empty_like(x))
    near(total, ref[1], tol, "with gradients")
    check(x, w, t)


@pytest.mark.parametrize("m,v", [(500, 2), (500, 3), (500, 5), (2000, 8), (900, 20), (2000, 64), (500, 65), (300, 200)])
def test_each_gradient_of_a_logit(m, v):
    """dz itself, which rows of the unit matrix in w hand on to dx: of the target within one rounding to bf16,
    2^-8, of the others within two, theirs and their exponentials', however few columns share a row."""
    gen = torch.Generator("cuda").manual_seed(v)
    slope = torch.randn(v, device="cuda", generator=gen).to(BF)
    x, w = blank(m, v + 1), blank(v, v + 1)
    x.zero_()
    x[:, 0] = torch.randn(m, device="cuda", generator=gen) * 3.0
    w.copy_(torch.cat([slope[:, None], torch.eye(v, device="cuda", dtype=BF)], 1))
    t = targets_of(m, v, 3)
    dx = blank(m, v + 1)
    za.zero_linear_cross_entropy(x, w, t, dx=dx, scale=torch.ones(m, device="cuda"))
    dz = o.cross_entropy(x, w, t, scale=torch.ones(m, device="cuda"))[4]
    half = torch.full_like(dz, 2.0 ** -7).scatter_(1, t[:, None], 2.0 ** -8)
    # (the exponentials' own error is 2^-17, as in tolerances; twice that for the sum's)
    near(dx[:, 1:], dz, (half * 1.01 + 3 * 2.0 ** -17) * dz.abs() + 1e-30, "dz")


def test_withheld_copies_of_wide_rows_are_reported():
    """Waits for one of several chains run out too; the next call is right."""
    m, k, v = 40, 1100, 515
    x, w, t = matrix(m, k, 1.0, 1), matrix(v, k, 0.05, 2), targets_of(m, v, 3)
    for kw in ({}, dict(dx=blank(m, k))):
        za.test_withhold_copies(True)
        try:
            za.zero_linear_cross_entropy(x, w, t, torch.zeros(m, device="cuda"), **kw)
            assert za.device_status() != za.ZERO_OK
        finally:
            za.test_withhold_copies(False)
    check(x, w, t)
