"""AdamW over a list of tensors, its 8-bit moments and the gradient norm on the GPU against the
64-bit statements of tests/train_oracle.py."""
import numpy as np
import pytest
import torch

import train_oracle as o
import zero_partitioned_mixed_adam_gb300 as za

pytestmark = pytest.mark.gpu

B1, B2, EPS, LR = 0.9, 0.95, 1e-8, 1e-3
SIZES = [1, 2, 31, 255, 256, 257, 0, 2047, 2048, 2049, 10000, 65536, 100003]


def cut(flat, sizes):
    return list(flat.split(sizes))


class Case:
    """A list of tensors on the host and the GPU; flat=True packs every buffer (so that
    tensors start at any element), "codes apart" all but the codes, else each has an
    allocation of its own."""

    def __init__(self, sizes, eight, f32, flat, seed=0, params=True):
        rng = np.random.default_rng(seed)
        self.sizes, self.eight, self.seed = sizes, eight, seed
        n = sum(sizes)
        spread = np.exp(rng.normal(0, 3, n))
        g = (rng.normal(0, 1e-3, n) * spread * (rng.random(n) > 0.1)).astype(np.float32)
        self.g = g if f32 else o.round_bf16(g)
        self.w = rng.normal(0, 0.02, n).astype(np.float32)
        self.m = (rng.normal(0, 3e-4, n) * spread).astype(np.float32)
        self.v = ((rng.normal(0, 1e-3, n) * spread) ** 2).astype(np.float32)
        self.decay = [0.1 * (i % 3) for i in range(len(sizes))]
        ends = np.cumsum([0] + sizes)
        self.cuts = [slice(a, b) for a, b in zip(ends[:-1], ends[1:])]
        if eight:
            half = np.full(n, 0x8000)
            self.mq = [o.encode(self.m[c], half[c], 4) for c in self.cuts]
            self.vq = [o.encode(self.v[c], half[c], 5) for c in self.cuts]
            self.m = np.concatenate([o.decode(*q, 4) for q in self.mq] or [np.zeros(0, np.float32)])
            self.v = np.concatenate([o.decode(*q, 5) for q in self.vq] or [np.zeros(0, np.float32)])

        def dev(x, dtype=None, packed=bool(flat)):
            t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
            t = t if dtype is None else t.to(dtype)
            return cut(t, sizes) if packed else [p.clone() for p in cut(t, sizes)]

        self.dg = dev(self.g, None if f32 else torch.bfloat16)
        self.dw = dev(self.w)
        self.dp = dev(np.zeros(n, np.float32), torch.bfloat16) if params else None
        kw = {}
        if eight:
            cat = lambda q, k, z: np.concatenate([x[k] for x in q] or [np.zeros(0, z)])  # noqa: E731
            self.dm, self.dv = (dev(cat(q, 0, np.uint8), packed=flat is True)
                                for q in (self.mq, self.vq))
            self.dms = [torch.from_numpy(s).cuda() for _, s in self.mq]
            self.dvs = [torch.from_numpy(s).cuda() for _, s in self.vq]
            kw = dict(m_scale=self.dms, v_scale=self.dvs)
        else:
            self.dm, self.dv = dev(self.m), dev(self.v)
        self.list = za.adamw_tensors(self.dg, self.dw, self.dm, self.dv, params=self.dp,
                                     weight_decay=self.decay, **kw)

    def step(self, t=7, seed=123, scale=None, **kw):
        ds = None if scale is None else torch.tensor([scale], dtype=torch.float32, device="cuda")
        za.zero_adamw_step(self.list, lr=LR, beta1=B1, beta2=B2, eps=EPS, t=t, seed=seed,
                           grad_scale=ds, **kw)
        torch.cuda.synchronize()
        g = self.g if scale is None else (self.g * np.float32(scale)).astype(np.float32)
        self.m, self.v = o.moments(g, self.m, self.v, B1, B2)
        self.w_old = self.w
        for i, c in enumerate(self.cuts):
            w64 = o.update(self.w[c], self.m[c], self.v[c], LR, self.decay[i], B1, B2, EPS, t)
            self.check_weights(i, c, w64, t)
            if self.eight:
                u = o.random_bits(seed, i, c.stop - c.start)
                for name, x, q, s, bits, r in (("m", self.m, self.dm, self.dms, 4, u >> np.uint64(16)),
                                               ("v", self.v, self.dv, self.dvs, 5, u & np.uint64(0xFFFF))):
                    codes, scales = o.encode(x[c], r, bits)
                    got = q[i].cpu().numpy()
                    assert np.array_equal(s[i].cpu().numpy(), scales, equal_nan=True), (name, i)
                    fine = np.repeat(~np.isnan(scales), o.BLOCK)[:len(codes)]
                    assert np.array_equal(got[fine], codes[fine]), (name, i)
                    x[c] = o.decode(got, scales, bits)
            else:
                assert np.array_equal(self.dm[i].cpu().numpy(), self.m[c], equal_nan=True), i
                assert np.array_equal(self.dv[i].cpu().numpy(), self.v[c], equal_nan=True), i

    def check_weights(self, i, c, w64, t):
        """The update is a quotient of binary32 values, each of its at most 12 operations (a
        scalar's rounding, a product, a root, a quotient) good to 2^-22; the last difference
        rounds to half a last place of the weight."""
        got = self.dw[i].cpu().numpy()
        keep = self.w[c].astype(np.float64) * (1.0 - LR * self.decay[i])
        fine = np.isfinite(w64)
        assert np.array_equal(np.isnan(got), np.isnan(w64))
        tol = 12 * 2.0 ** -22 * np.abs(w64 - keep) + 2.0 ** -23 * (np.abs(keep) + np.abs(w64)) + 1e-44
        assert (np.abs(got[fine] - w64[fine]) <= tol[fine]).all()
        if self.dp is not None:
            p = self.dp[i].float().cpu().numpy()
            assert np.array_equal(p, o.round_bf16(got), equal_nan=True)
        self.w = np.array(self.w)
        self.w[c] = got


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("flat", [False, True])
def test_steps(eight, f32, flat):
    case = Case(SIZES, eight, f32, flat)
    case.step(t=7, seed=123)
    case.step(t=8, seed=2 ** 32 - 1, scale=0.37)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("f32", [False, True])
def test_every_start_within_16_bytes(eight, f32):
    """Tensors that begin 0 to 7 elements past a 16-byte boundary, from shorter than that to
    several tiles."""
    sizes = [2049] * 9 + [1, 6, 7, 257, 255, 1025, 513, 33, 4099]
    starts = np.cumsum([0] + sizes)
    assert set(starts[:9] % 8) == set(range(8))
    case = Case(sizes, eight, f32, "codes apart")
    case.step(t=7, seed=9)
    case.step(t=8, seed=10, scale=0.37)
    case = Case(sizes, eight, f32, "codes apart", params=False)
    case.step(t=7, seed=9)


@pytest.mark.parametrize("eight", [False, True])
def test_without_parameters_and_one_by_one(eight):
    case = Case([5, 700], eight, True, False, params=False)
    case.step(t=1)
    assert Case([], eight, False, False).list.arr is not None
    za.zero_adamw_step(Case([], eight, False, False).list, lr=LR, t=1)
    za.zero_adamw_step(Case([0, 0], eight, False, False).list, lr=LR, t=1)


@pytest.mark.parametrize("eight", [False, True])
def test_more_tensors_than_one_launch_holds(eight):
    rng = np.random.default_rng(5)
    case = Case([int(x) for x in rng.integers(0, 700, 1200)], eight, False, True)
    case.step()


@pytest.mark.parametrize("eight", [False, True])
def test_infinities_and_nan(eight):
    """A non-finite gradient reaches its own weight (and, in 8 bits, its block's moments)
    and nothing else."""
    case = Case([1000, 600], eight, True, False)
    for i, x in ((3, np.nan), (300, np.inf), (1100, -np.inf)):
        case.g[i] = x
        (case.dg[0] if i < 1000 else case.dg[1])[i if i < 1000 else i - 1000] = float(x)
    case.step()
    bad = np.isnan(case.w)
    assert set(np.flatnonzero(bad)) == {3, 300, 1100}
    if eight:
        for i in (0, 1):
            blocks = np.isnan(case.dms[i].cpu().numpy())
            assert blocks.tolist() == [[True, True, False, False], [True, False, False]][i]


@pytest.mark.parametrize("magnitude", [0.0, 1e-30, 1e-38, 1e-42, 1e15])
def test_8bit_range(magnitude):
    """Zero, denormal and very large gradients: codes and scales as defined."""
    case = Case([513], True, True, False)
    rng = np.random.default_rng(1)
    case.g[:] = (rng.normal(0, 1, 513) * magnitude).astype(np.float32)
    case.dg[0].copy_(torch.from_numpy(case.g))
    for t in (case.dm[0], case.dv[0], case.dms[0], case.dvs[0]):
        t.zero_()
    case.m[:], case.v[:] = 0.0, 0.0
    case.step(t=1)
    case.step(t=2)


def test_8bit_rounding_is_unbiased():
    """Encoding the same moments with 400 seeds: each code is one of the two around the
    value, and the mean of the values is the value within 6 standard errors of it."""
    n, seeds = 256, 400
    rng = np.random.default_rng(2)
    m0 = (rng.normal(0, 1, n) * np.exp(rng.normal(0, 2, n))).astype(np.float32)
    mean, sq = np.zeros(n), np.zeros(n)
    for seed in range(seeds):
        # beta1 = 0: the new m is g itself
        g = torch.from_numpy(m0).cuda()
        w, codes = torch.zeros(n, device="cuda"), [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.zeros(1, device="cuda") for _ in range(2)]
        lst = za.adamw_tensors([g], [w], [codes[0]], [codes[1]], m_scale=[scales[0]], v_scale=[scales[1]])
        za.zero_adamw_step(lst, lr=0.0, beta1=0.0, t=1, seed=seed)
        x = o.decode(codes[0].cpu().numpy(), scales[0].cpu().numpy(), 4).astype(np.float64)
        mean += x / seeds
        sq += (x - m0) ** 2 / seeds
    step = np.maximum(np.exp2(np.floor(np.log2(np.abs(m0))) - 3), float(scales[0]) * 2.0 ** -17)
    assert (np.sqrt(sq) <= step).all()
    assert (np.abs(mean - m0) <= 6 * step / 2 / np.sqrt(seeds)).all()


def test_8bit_values_that_do_not_change_are_held():
    """A value that is a code's is held exactly whatever the seed: beta = 0 and the decoded
    moments as gradients give the same codes again."""
    case = Case([1000], True, True, False)
    g = torch.from_numpy(case.m).cuda()
    lst = za.adamw_tensors([g], case.dw, case.dm, case.dv, m_scale=case.dms, v_scale=case.dvs)
    before = case.dm[0].clone()
    for seed in (1, 2, 3):
        za.zero_adamw_step(lst, lr=0.0, beta1=0.0, t=1, seed=seed)
        assert torch.equal(o_value(case.dm[0], case.dms[0]), o_value(before, case.dms[0]))


def o_value(codes, scales):
    return torch.from_numpy(o.decode(codes.cpu().numpy(), scales.cpu().numpy(), 4))


@pytest.mark.parametrize("sizes", [[1], [255, 256, 257, 0, 5000], SIZES, [300] * 700])
def test_moment_values(sizes):
    case = Case(sizes, True, False, True)
    outs = [[torch.full((n,), 7.0, device="cuda") for n in sizes] for _ in range(2)]
    za.zero_adamw_state_f32(case.list, outs[0], outs[1])
    for out, x in zip(outs, (case.m, case.v)):
        assert np.array_equal(torch.cat(out).cpu().numpy(), x)
    za.zero_adamw_state_f32(case.list, None, outs[0])
    assert np.array_equal(torch.cat(outs[0]).cpu().numpy(), case.v)


def test_same_bits_every_time_on_any_stream():
    a, b = Case(SIZES, True, False, True), Case(SIZES, True, False, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a.step(seed=9)
    b.step(seed=9, stream=side)
    for x, y in zip(a.dm + a.dv + a.dw + a.dms, b.dm + b.dv + b.dw + b.dms):
        assert torch.equal(x, y)


# ------------------------------------------------------------------------------- norm

def norm_of(grads, most=1.0, ws=None):
    out = torch.full((2,), -1.0, device="cuda")
    ws = za.grad_norm_workspace() if ws is None else ws
    za.zero_grad_norm(za.grad_list(grads), out, max_norm=most, workspace=ws)
    return [float(x) for x in out.cpu()]


def check_norm(grads, most=1.0, ws=None):
    """fp32 runs of 64 squares (each sum good to 64 roundings of 2^-24), fp64 from there, one
    rounding of the root: 2^-18 of the sum at the very most, half of that of the norm."""
    norm, coef = norm_of(grads, most, ws)
    want = np.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))
    assert abs(norm - want) <= 2.0 ** -19 * want
    # coef in binary32 from the norm: an addition and a quotient
    assert abs(coef - min(1.0, most / (norm + 1e-6))) <= 2.0 ** -22
    return norm, coef


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sizes", [[1], [0, 7, 0], [16383, 16384, 16385], [3, 5, 100003, 1, 65537], [33] * 2500])
def test_norm(dtype, sizes):
    gen = torch.Generator("cuda").manual_seed(3)
    flat = torch.empty(sum(sizes) + 3, device="cuda").normal_(0, 1e-2, generator=gen).to(dtype)
    ws = za.grad_norm_workspace()
    for first in (0, 1, 3):
        grads = cut(flat[first:first + sum(sizes)], sizes)
        a = check_norm(grads, 1e-3, ws)
        assert check_norm(grads, 1e-3, ws) == a     # the same bits, and the workspace is ready again
    assert check_norm(cut(flat[:sum(sizes)], sizes), 1e6)[1] == 1.0


def test_norm_of_nothing_and_of_what_is_not_finite():
    assert norm_of([]) == [0.0, 1.0]
    g = torch.ones(5000, device="cuda")
    g[4999] = float("inf")
    assert norm_of([g]) == [float("inf"), 0.0]
    g[17] = float("nan")
    norm, coef = norm_of([g])
    assert np.isnan(norm) and np.isnan(coef)
    assert norm_of([torch.zeros(77, device="cuda")], 0.0)[0] == 0.0


def test_norm_clips_the_step():
    case = Case(SIZES, False, False, True)
    out, ws = torch.empty(2, device="cuda"), za.grad_norm_workspace()
    za.zero_grad_norm(case.list, out, max_norm=1e-2, workspace=ws)
    coef = np.float32(out[1].item())
    assert 0.0 < coef < 1.0
    za.zero_adamw_step(case.list, lr=LR, beta1=B1, beta2=B2, eps=EPS, t=3, grad_scale=out[1:])
    m, _ = o.moments((case.g * coef).astype(np.float32), case.m, case.v, B1, B2)
    assert np.array_equal(torch.cat(case.dm).cpu().numpy(), m)


def test_steps_and_norm_in_a_graph():
    """Captured once their kernels have run, replayed twice: the same as two calls."""
    a, b = Case([1000, 3, 5000], True, False, True), Case([1000, 3, 5000], True, False, True)
    out, ws = torch.empty(2, device="cuda"), za.grad_norm_workspace()

    def both(case):
        za.zero_grad_norm(case.list, out, max_norm=1e-2, workspace=ws)
        za.zero_adamw_step(case.list, lr=LR, beta1=B1, beta2=B2, t=5, seed=4, grad_scale=out[1:])

    both(a)
    both(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(b)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(a.dm + a.dv + a.dw, b.dm + b.dv + b.dw):
        assert torch.equal(x, y)


def test_more_than_32_bits_of_elements():
    """One 8-bit tensor of 2^32 + 1000 elements: offsets past 32 bits, and the random bits
    of the elements past 2^32.  The gradient is zero but at the two ends."""
    n = 2 ** 32 + 1000
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(n, device="cuda")
    codes = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(-(-n // 256), device="cuda") for _ in range(2)]
    rng = np.random.default_rng(0)
    tail = o.round_bf16(rng.normal(0, 1, 1000).astype(np.float32))
    g[:1000] = torch.from_numpy(tail).cuda()
    g[-1000:] = torch.from_numpy(tail).cuda()
    lst = za.adamw_tensors([g], [w], [codes[0]], [codes[1]], m_scale=[scales[0]], v_scale=[scales[1]])
    za.zero_adamw_step(lst, lr=LR, beta1=B1, beta2=B2, t=1, seed=77)
    m, _ = o.moments(tail, np.zeros(1000, np.float32), np.zeros(1000, np.float32), B1, B2)
    key = o.pcg((o.pcg(np.uint64(77))) & np.uint64(0xFFFFFFFF))
    for lo, high in ((0, 0), (n - 1000, 1)):
        k = (int(key) + high * 0x9E3779B9) & 0xFFFFFFFF
        u = o.pcg((np.arange(1000, dtype=np.uint64) + np.uint64(k)) & np.uint64(0xFFFFFFFF))
        want, _ = o.encode(m, u >> np.uint64(16), 4)
        got = codes[0][lo:lo + 1000].cpu().numpy()
        # (2^32 is a multiple of 256: the tail's blocks start where the head's do, the last is cut)
        assert np.array_equal(got[:768], want[:768]) and np.array_equal(got[768:], want[768:])
    assert not bool(codes[0][1024:10 ** 6].any())
    out = torch.empty(2, device="cuda")
    za.zero_grad_norm(lst, out, max_norm=1.0, workspace=za.grad_norm_workspace())
    want = np.sqrt(2 * (tail.astype(np.float64) ** 2).sum())
    assert abs(float(out[0]) - want) <= 2.0 ** -19 * want
