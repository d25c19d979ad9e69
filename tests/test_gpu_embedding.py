"""Embedding lookup and its gradient on the GPU against 64 bits."""
import pytest
import torch

import model_oracle as o
import zero_partitioned_mixed_adam_gb300 as za

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64

# rows, width, vocabulary: ones; around a warp's and a slice's columns; odd; more tokens than
# are sorted at one time (4,096 a class); wide
SHAPES = [(1, 1, 1), (1, 2048, 50), (2, 7, 3), (33, 8, 100), (50, 255, 17), (64, 256, 1000), (100, 257, 9),
          (129, 775, 513), (300, 1024, 64), (700, 1032, 333), (40, 5000, 20), (900, 80, 20000)]


def matrix(rows, cols, sigma, seed, pitch=0, offset=0, dtype=BF):
    gen = torch.Generator("cuda").manual_seed(seed)
    flat = torch.empty(offset + rows * (cols + pitch), device="cuda").normal_(0, sigma, generator=gen).to(dtype)
    return flat[offset:].view(rows, cols + pitch)[:, :cols]


def blank(rows, cols, dtype=BF, pitch=0, offset=0):
    flat = torch.full((offset + rows * (cols + pitch),), 7.0, dtype=dtype, device="cuda")
    return flat[offset:].view(rows, cols + pitch)[:, :cols]


def ids_of(rows, vocab, seed, dtype=torch.int64):
    """A quarter of them one token, the others evenly."""
    gen = torch.Generator("cuda").manual_seed(seed)
    ids = torch.randint(0, vocab, (rows,), device="cuda", generator=gen)
    return torch.where(torch.rand(rows, device="cuda", generator=gen) < 0.25, vocab // 2, ids).to(dtype)


def untouched(view):
    flat = view._base
    view.fill_(7.0)
    assert (flat == 7.0).all()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("ids,scale,pitch,offset", [(torch.int64, 1.0, 0, 0), (torch.int32, 22.6, 8, 8),
                                                    (torch.int64, -0.3, 1, 3)])
def test_lookup(shape, ids, scale, pitch, offset):
    m, d, v = shape
    table, y, i = matrix(v, d, 1.0, 1, pitch, offset), blank(m, d, BF, pitch, offset), ids_of(m, v, 2, ids)
    za.zero_embedding_forward(i, table, y, scale=scale)
    # the product in fp32, as torch has it too, and one rounding: the same bits
    assert torch.equal(y, (table.float() * torch.tensor(scale, dtype=F32, device="cuda")).to(BF)[i.long()])
    untouched(y)


def check(dy, ids, dtable, *, scale=1.0, padding=None, add=False, **kw):
    before = dtable.to(F64) if add else torch.zeros(dtable.shape, dtype=F64, device="cuda")
    za.zero_embedding_backward(dy, ids, dtable, scale=scale, padding=padding, accumulate=add, **kw)
    want = o.embedding_grad(dy, ids, dtable.shape[0], scale, padding) + before
    size = o.embedding_grad(dy.abs(), ids, dtable.shape[0], abs(scale), padding)
    count = o.embedding_grad(torch.ones_like(dy[:, :1]), ids, dtable.shape[0], 1.0, padding)
    # chains of 64 rows, a chain of those, 8 warps' (few tokens: 16 and 8 blocks'), the scale and what
    # is added: 2^-24 each of the sum of magnitudes; then the rounding to the type
    steps = torch.clamp(count, max=64) + count / 64 / 8 + 28
    half = 2.0 ** -8 if dtable.dtype == BF else 2.0 ** -24
    tol = steps * 2.0 ** -24 * (size + before.abs())
    got = dtable.to(F64)
    assert torch.isfinite(got).all()
    assert ((got - want).abs() <= tol + half * (want.abs() + tol)).all()
    assert (got == before)[(count == 0).expand_as(got)].all()      # rows of no token, to the bit


# few tokens, whose rows several blocks share: around the runs of rows and what is added at a time;
# tokens of no row; and as many tokens as there are blocks of their own for, and one more
FEW = [(9000, 64, 2), (5000, 775, 3), (20000, 260, 1), (3000, 2048, 19), (511, 8, 304), (513, 8, 305), (4097, 100, 608),
       (4097, 100, 609), (8192, 16, 5)]


@pytest.mark.parametrize("shape", FEW)
@pytest.mark.parametrize("dtype,add,ids,pitch,offset", [
    (BF, False, torch.int64, 0, 0), (F32, True, torch.int32, 8, 8), (BF, True, torch.int64, 1, 3),
    (F32, False, torch.int32, 5, 1)])
def test_gradient_of_few_tokens(shape, dtype, add, ids, pitch, offset):
    m, d, v = shape
    dy, i = matrix(m, d, 1.0, 1, pitch, offset), ids_of(m, v, 2, ids)
    for padding in (None, 0, v // 2):
        dtable = matrix(v, d, 1.0, 3, pitch, offset, dtype) if add else blank(v, d, dtype, pitch, offset)
        check(dy, i, dtable, scale=1.5, add=add, padding=padding)
        again = matrix(v, d, 1.0, 3, pitch, offset, dtype) if add else blank(v, d, dtype, pitch, offset)
        za.zero_embedding_backward(dy, i, again, scale=1.5, padding=padding, accumulate=add)
        assert torch.equal(again, dtable)
        if not add:
            untouched(dtable)
    i[m // 3:] = v                # ids outside the table, and of the rest all one token
    i[:m // 3] = v - 1
    dtable = matrix(v, d, 1.0, 3, pitch, offset, dtype) if add else blank(v, d, dtype, pitch, offset)
    check(dy, i, dtable, scale=1.5, add=add)


@pytest.mark.parametrize("width", [1, 7, 8, 100, 255, 256, 257, 263, 513])
@pytest.mark.parametrize("offset", [0, 1, 2, 3, 4, 5, 6, 7])
def test_gradients_rows_at_every_address(width, offset):
    """Rows that begin at every 2-byte place of a 16-byte vector, among values that are not theirs."""
    flat = torch.full((40 * (width + 3) + 16,), float("nan"), dtype=BF, device="cuda")
    for v in (2, 400):
        dy = flat[offset:offset + 40 * (width + 3)].view(40, width + 3)[:, :width]
        dy.copy_(matrix(40, width, 1.0, 1))
        check(dy, ids_of(40, v, 2), blank(v, width))


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype,add,ids,pitch,offset", [
    (BF, False, torch.int64, 0, 0), (F32, False, torch.int32, 0, 0), (F32, True, torch.int64, 8, 8),
    (BF, True, torch.int32, 1, 3), (F32, False, torch.int64, 3, 1)])
def test_gradient(shape, dtype, add, ids, pitch, offset):
    m, d, v = shape
    dtable = matrix(v, d, 1.0, 3, pitch, offset, dtype) if add else blank(v, d, dtype, pitch, offset)
    check(matrix(m, d, 1.0, 1, pitch, offset), ids_of(m, v, 2, ids), dtable, scale=1.5, add=add)
    if not add:
        untouched(dtable)


@pytest.mark.parametrize("rows,vocab", [(3000, 1), (3000, 5), (20000, 2), (40000, 400), (30000, 30000)])
def test_common_tokens(rows, vocab):
    """Every row one token; more rows of a token, and of a class of tokens, than are sorted at
    one time."""
    d = 300
    ids = ids_of(rows, vocab, 2)
    check(matrix(rows, d, 1.0, 1), ids, blank(vocab, d))
    check(matrix(rows, d, 1.0, 1), torch.full_like(ids, vocab - 1), blank(vocab, d, F32))


def test_wide_tables():
    """So wide that a block has every token: 304 slices of 256 columns and more."""
    check(matrix(9, 80000, 1.0, 1), ids_of(9, 5000, 2), blank(5000, 80000))


@pytest.mark.parametrize("add", [False, True])
def test_ids_without_a_gradient(add):
    m, d, v = 500, 264, 40
    ids = ids_of(m, v, 2)
    ids[3], ids[70], ids[71] = -1, v, 2 ** 40
    dy = matrix(m, d, 1.0, 1)
    dy[3] = float("nan")                       # nothing of these rows counts
    dy[ids == 7] = float("inf")
    for padding in (None, 7, -100):
        if padding != 7:
            dy[ids == 7] = 1.0
        check(dy.clone(), ids, matrix(v, d, 1.0, 5) if add else blank(v, d), padding=padding, add=add)
        dy[ids == 7] = float("inf")


def test_lookup_of_ids_outside_the_table():
    table, y = matrix(10, 100, 1.0, 1), blank(5, 100)
    za.zero_embedding_forward(torch.tensor([0, -1, 9, 10, 2 ** 33], device="cuda"), table, y)
    assert torch.equal(y[0], table[0]) and torch.equal(y[2], table[9])
    assert y[[1, 3, 4]].isnan().all()


def test_no_rows():
    ids, none, dtable = torch.empty(0, dtype=torch.int64, device="cuda"), blank(1, 16)[:0], blank(9, 16)
    za.zero_embedding_forward(ids, dtable, none)
    za.zero_embedding_backward(none, ids, dtable, accumulate=True)
    assert (dtable == 7.0).all()
    za.zero_embedding_backward(none, ids, dtable)
    assert not dtable.any()


def test_the_same_bits_every_time_and_on_another_stream():
    m, d, v = 5000, 520, 700
    dy, ids = matrix(m, d, 1.0, 1), ids_of(m, v, 2)
    want = blank(v, d, F32)
    za.zero_embedding_backward(dy, ids, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side, None):
        got = blank(v, d, F32)
        side.wait_stream(torch.cuda.current_stream())
        za.zero_embedding_backward(dy, ids, got, stream=stream)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)
    graph, y = torch.cuda.CUDAGraph(), blank(m, d)
    with torch.cuda.graph(graph):
        za.zero_embedding_forward(ids, want.to(BF), y)
        za.zero_embedding_backward(dy, ids, got)
    ids.copy_(ids_of(m, v, 9))
    graph.replay()
    check(dy, ids, want)
    assert torch.equal(got, want)
