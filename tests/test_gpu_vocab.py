"""GPU parity of the embedding and of the linear cross entropy with their gradients, against the float64
formulas of oracle/vocab.py, whose docstring derives the bounds."""
import threading

import pytest
import torch

import fp32_row_reduction_gb300 as tr
from oracle import vocab

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
IGNORE = -100


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tr.load()


def gen(seed):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    return g


def randn(g, shape, dtype, scale=1.0, offset=0):
    """A contiguous tensor that starts `offset` elements into its allocation."""
    n = 1
    for s in shape:
        n *= s
    t = torch.empty(n + offset, device=DEV, dtype=dtype)
    t.copy_(torch.randn(n + offset, generator=g, device=DEV) * scale)
    return t[offset:].view(shape)


def close(got, want, dtype=None):
    v, err = want
    assert got.shape == v.shape
    dtype = dtype or got.dtype
    bad = (got.double() - v).abs() - vocab.rounded(v, err, dtype)
    bad = torch.where(torch.isnan(bad), torch.full_like(bad, float("inf")), bad)
    assert bad.numel() == 0 or float(bad.max()) <= 0.0, (float(bad.max()), int((bad > 0).sum()), bad.numel())


def same(a, b):
    """Equal bits."""
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---- embedding ------------------------------------------------------------------------

EMBED = [(1, 1, 1), (1, 100, 4096), (3, 5, 7), (48, 5003, 5120), (300, 17, 65), (257, 1000, 1537), (1000, 50257, 128), (33, 64, 8), (5, 9, 2056)]


@pytest.mark.parametrize("tokens,v,cols", EMBED)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset", [0, 1])
def test_embedding(tokens, v, cols, dtype, offset):
    g, dt = gen(tokens + cols), DTYPES[dtype]
    table = randn(g, (v, cols), dt, offset=offset)
    ids = torch.randint(-2, v + 2, (tokens,), generator=g, device=DEV)
    close(tr.embedding(ids, table, scale=0.3), vocab.embedding(ids, table, 0.3))
    guard = torch.full((tokens * cols + 64,), 7.0, device=DEV, dtype=dt)  # what is behind the rows stays
    out = guard[3:3 + tokens * cols].view(tokens, cols)
    tr.embedding(ids, table, out=out)
    inside = (ids >= 0) & (ids < v)
    want = torch.where(inside[:, None], table[ids.clamp(0, v - 1)], torch.zeros((), device=DEV, dtype=dt))
    assert torch.equal(out, want)  # a scale of 1 changes nothing
    assert bool((guard[:3] == 7).all()) and bool((guard[3 + tokens * cols:] == 7).all())


def test_embedding_shapes_and_values():
    g = gen(1)
    table = randn(g, (50, 24), torch.bfloat16)
    table[7] = float("inf")
    table[8] = float("nan")
    ids = torch.tensor([[[7, 1], [8, -1]], [[49, 50], [1 << 40, -(1 << 62)]]], device=DEV)
    y = tr.embedding(ids, table, scale=2.0)
    assert y.shape == (2, 2, 2, 24) and bool(torch.isinf(y[0, 0, 0]).all()) and bool(torch.isnan(y[0, 1, 0]).all())
    assert torch.equal(y[0, 0, 1], 2 * table[1]) and torch.equal(y[1, 0, 0], 2 * table[49])
    assert not y[0, 1, 1].any() and not y[1, 0, 1].any() and not y[1, 1].any()
    assert tr.embedding(ids[:0], table).shape == (0, 2, 2, 24)
    with pytest.raises(TypeError):
        tr.embedding(ids.int(), table)
    with pytest.raises(ValueError):
        tr.embedding(ids, table[:, :8])
    with pytest.raises(ValueError):
        tr.embedding(ids[:, :, 0], table)


# ---- the embedding's gradient -----------------------------------------------------------

def token_ids(g, n, v, spread):
    if spread == "one":
        return torch.full((n,), v // 2, device=DEV, dtype=torch.int64)
    if spread == "runs":  # segments of every length about the tile's and the longest short one's
        lengths = [1, 31, 32, 33, 63, 64, 65, 95, 96, 97, 128, 129, 2, 1, 200]
        ids = torch.cat([torch.full((lengths[i % len(lengths)],), (3 * i) % v, dtype=torch.int64) for i in range(1 + n // 30)])[:n]
        return ids[torch.randperm(n, generator=torch.Generator().manual_seed(5))].to(DEV)
    if spread == "outside":
        return torch.randint(-v, 0, (n,), generator=g, device=DEV)
    ids = torch.randint(0, v, (n,), generator=g, device=DEV)
    if spread == "padded":
        ids[torch.rand(n, generator=g, device=DEV) < 0.5] = -1
        ids[::7] = v
    return ids


GRADS = [(1, 1, 1, "even"), (1, 50257, 64, "even"), (48, 5003, 512, "even"), (64, 3, 40, "one"), (65, 3, 40, "one"), (97, 300, 1537, "padded"),
         (1000, 37, 256, "runs"), (3000, 999, 136, "runs"), (2500, 999, 33, "runs"), (5000, 5003, 72, "padded"), (16384, 211, 24, "even"),
         (16385, 211, 24, "runs"), (40000, 70001, 16, "padded"), (33000, 5, 8, "one"), (20000, (1 << 24) + 3, 1, "even"), (100, 7, 300, "outside"),
         (17000, 300, 9, "outside")]


@pytest.mark.parametrize("tokens,v,cols,spread", GRADS)
@pytest.mark.parametrize("dtype,grad", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
def test_embedding_backward(tokens, v, cols, spread, dtype, grad):
    g, dt, gt = gen(tokens + v), DTYPES[dtype], DTYPES[grad]
    dy = randn(g, (tokens, cols), dt)
    ids = token_ids(g, tokens, v, spread)
    dy[(ids < 0) | (ids >= v)] = float("nan")  # padding holds anything
    guard = torch.full((v * cols + 64,), 7.0, device=DEV, dtype=gt)
    dtable = guard[32:32 + v * cols].view(v, cols)
    dtable.fill_(float("nan"))
    tr.embedding_backward(dy, ids, scale=0.7, dtable=dtable)
    close(dtable, vocab.embedding_backward(dy, ids, v, 0.7))
    assert bool((guard[:32] == 7).all()) and bool((guard[32 + v * cols:] == 7).all())
    again = torch.empty_like(dtable)
    tr.embedding_backward(dy, ids, scale=0.7, dtable=again)
    assert same(again, dtable)
    base = randn(g, (v, cols), gt)
    base[v - 1] = float("nan")  # rows that no token has are left alone
    total = base.clone()
    tr.embedding_backward(dy, ids, scale=0.7, dtable=total, accumulate=True)
    has = torch.zeros(v, dtype=torch.bool, device=DEV)
    has[ids[(ids >= 0) & (ids < v)]] = True
    assert same(total[~has], base[~has])
    want, err = vocab.embedding_backward(dy, ids, v, 0.7, base)
    keep = has & ~torch.isnan(base).any(1)
    close(total[keep], (want[keep], err[keep]))


@pytest.mark.parametrize("offset", [1, 4])
@pytest.mark.parametrize("dtype", DTYPES)
def test_embedding_backward_alignments(offset, dtype):
    g, dt = gen(offset), DTYPES[dtype]
    dy = randn(g, (700, 64), dt, offset=offset)
    ids = token_ids(g, 700, 90, "runs")
    flat = torch.empty(90 * 64 + offset, device=DEV, dtype=dt)
    dtable = flat[offset:].view(90, 64)
    tr.embedding_backward(dy, ids, dtable=dtable)
    close(dtable, vocab.embedding_backward(dy, ids, 90, 1.0))
    assert same(dtable, tr.embedding_backward(dy.clone(), ids, 90))  # whatever the alignment


@pytest.mark.parametrize("dtype,grad", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
def test_adding_to_a_table_rounds_once(dtype, grad):
    """base + scale sum is one rounding of binary32 (and one of the type), whatever the alignment: the bits are the same."""
    g, dt, gt = gen(14), DTYPES[dtype], DTYPES[grad]
    dy, base = randn(g, (900, 64), dt), randn(g, (70, 64), gt)
    ids = token_ids(g, 900, 70, "runs")
    want = base.clone()
    tr.embedding_backward(dy, ids, scale=0.7, dtable=want, accumulate=True)
    for offset in (1, 4):
        flat = torch.empty(70 * 64 + offset, device=DEV, dtype=gt)
        table = flat[offset:].view(70, 64)
        table.copy_(base)
        tr.embedding_backward(dy, ids, scale=0.7, dtable=table, accumulate=True)
        assert same(table, want)
    # a single token's sum is its row: its product with the scale is exact in float64, whose sum is rounded far below binary32
    one = base.float().clone()
    tr.embedding_backward(dy[:1], ids[:1], scale=0.7, dtable=one, accumulate=True)
    exact = base[ids[0]].double() + vocab.f32(0.7) * dy[0].double()
    assert torch.equal(one[ids[0]], exact.float())


def test_embedding_backward_arguments():
    g = gen(0)
    dy, ids = randn(g, (4, 6, 16), torch.float16), torch.randint(0, 9, (4, 6), generator=g, device=DEV)
    dtable = tr.embedding_backward(dy, ids, 9)
    assert dtable.shape == (9, 16) and dtable.dtype == torch.float16
    close(dtable, vocab.embedding_backward(dy, ids, 9, 1.0))
    empty = tr.embedding_backward(dy[:0], ids[:0], 9, dtable=torch.full((9, 16), 3.0, device=DEV))
    assert not empty.any()
    kept = tr.embedding_backward(dy[:0], ids[:0], dtable=torch.full((9, 16), 3.0, device=DEV), accumulate=True)
    assert bool((kept == 3).all())
    with pytest.raises(ValueError):
        tr.embedding_backward(dy, ids)
    with pytest.raises(ValueError):
        tr.embedding_backward(dy, ids, 9, accumulate=True)
    with pytest.raises(ValueError):
        tr.embedding_backward(dy, ids[:3], 9)
    with pytest.raises(TypeError):
        tr.embedding_backward(dy, ids, dtable=torch.zeros(9, 16, device=DEV, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        tr.embedding_backward(dy, ids, 9, dtable=torch.zeros(8, 16, device=DEV))
    with pytest.raises(tr.TrError):
        tr.embedding_backward(dy, ids, 9, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


# ---- the loss ---------------------------------------------------------------------------

def loss_inputs(rows, cols, v, dtype, seed=0, ignored=0.0, offset=0, outside=False):
    g, dt = gen(seed + rows + cols + v), DTYPES[dtype]
    hidden = randn(g, (rows, cols), dt, offset=offset)
    weight = randn(g, (v, cols), dt, 1.5 / cols ** 0.5, offset=offset if cols % 8 else 0)
    labels = torch.randint(0, v, (rows,), generator=g, device=DEV)
    if outside and rows > 2:
        labels[0], labels[1], labels[2] = v, -1, 1 << 40
    gone = torch.rand(rows, generator=g, device=DEV) < ignored
    labels[gone] = IGNORE
    hidden[gone] = float("nan")  # padding holds anything
    dloss = torch.rand(rows, generator=g, device=DEV) / rows
    dlse = torch.randn(rows, generator=g, device=DEV) / rows
    dloss[gone] = float("nan")
    return hidden, weight, labels, dloss, dlse


def check_loss(hidden, weight, labels, dloss, dlse, scale=1.0, **kw):
    losses, lse = tr.linear_cross_entropy(hidden, weight, labels, logit_scale=scale, **kw)
    ignore = kw.get("ignore_label", IGNORE)
    want, want_lse = vocab.linear_cross_entropy(hidden, weight, labels, scale, ignore)
    close(losses, want)
    close(lse, want_lse)
    dh, dw = tr.linear_cross_entropy_backward(hidden, weight, labels, lse, dloss, dlse, logit_scale=scale, **kw)
    want_h, want_w = vocab.linear_cross_entropy_backward(hidden, weight, labels, lse, dloss, dlse, scale, ignore)
    close(dh, want_h)
    close(dw, want_w)
    assert tr.tr_last_device_error() == tr.TR_OK
    return losses, lse, dh, dw


LOSSES = [(1, 1, 1), (1, 8, 2), (2, 7, 3), (1, 64, 5003), (3, 65, 255), (37, 1537, 1000), (48, 512, 257), (128, 96, 256), (129, 1024, 64),
          (255, 33, 65), (256, 64, 513), (257, 136, 1000), (300, 264, 127), (513, 72, 2049), (700, 1000, 100), (1, 4096, 600), (1030, 16, 16)]


@pytest.mark.parametrize("rows,cols,v", LOSSES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_loss(rows, cols, v, dtype):
    hidden, weight, labels, dloss, dlse = loss_inputs(rows, cols, v, dtype, outside=rows > 50)
    check_loss(hidden, weight, labels, dloss, dlse)
    check_loss(hidden, weight, labels, None, None, scale=-0.7)


@pytest.mark.parametrize("rows,cols,v", [(37, 40, 300), (600, 129, 700), (1000, 64, 90), (1500, 129, 300)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("ignored", [0.3, 0.97, 1.0])
def test_rows_without_a_loss(rows, cols, v, dtype, ignored):
    hidden, weight, labels, dloss, dlse = loss_inputs(rows, cols, v, dtype, ignored=ignored, offset=1)
    losses, lse, dh, dw = check_loss(hidden, weight, labels, dloss, dlse)
    gone = labels == IGNORE
    assert not losses[gone].any() and not lse[gone].any() and not dh[gone].any()
    # one of the vocabulary's own labels as the one to leave out
    hidden, weight, labels, dloss, dlse = loss_inputs(rows, cols, v, dtype, seed=1)
    labels[rows // 3:] = 5
    check_loss(hidden, weight, labels, dloss, dlse, ignore_label=5)


@pytest.mark.parametrize("rows,cols,v", [(4, 8, 600_000), (1, 24, 1_100_000), (40_000, 16, 5003)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_loss_in_pieces(rows, cols, v, dtype):
    check_loss(*loss_inputs(rows, cols, v, dtype, ignored=0.2 if rows > 4 else 0.0))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,cols,v", [(5, 64, 999), (300, 520, 3000)])
def test_exact_logits(rows, cols, v, dtype):
    """Inputs of a few bits, so that every logit is exact in any order of the sum: what is left are the exponentials
    and logarithms, 2^-20 and a few u of the numbers they meet."""
    g, dt = gen(rows), DTYPES[dtype]
    hidden = torch.randint(-2, 3, (rows, cols), generator=g, device=DEV).to(dt)
    weight = (torch.randint(-3, 4, (v, cols), generator=g, device=DEV) / 32).to(dt)
    labels = torch.randint(0, v, (rows,), generator=g, device=DEV)
    losses, lse = tr.linear_cross_entropy(hidden, weight, labels)
    z = hidden.double() @ weight.double().T
    want = torch.logsumexp(z, 1)
    bound = 2.0 ** -20 + (64 + v / 64) * vocab.U + 8 * vocab.U * (want.abs() + z.abs().amax(1))
    assert bool(((lse.double() - want).abs() <= bound).all())
    assert bool(((losses.double() - (want - z.gather(1, labels[:, None])[:, 0])).abs() <= 2 * bound).all())


def test_certain_rows():
    """Rows whose label has all of the probability: the loss is as small as it is, not a difference of large numbers."""
    rows, cols, v = 64, 64, 300
    hidden = torch.zeros(rows, cols, device=DEV, dtype=torch.bfloat16)
    weight = torch.zeros(v, cols, device=DEV, dtype=torch.bfloat16)
    hidden[:, 0] = torch.arange(8, 8 + rows, device=DEV).to(torch.bfloat16)
    weight[3, 0] = 1.0
    labels = torch.full((rows,), 3, device=DEV)
    losses, lse = tr.linear_cross_entropy(hidden, weight, labels)
    x = hidden[:, 0].double()
    want = torch.log1p((v - 1) * torch.exp(-x))
    # The sum is 1 + s < 2, and s is off by 2^-20 and 4 u x of itself. An addition whose partial sum has the 1 in it rounds by
    # at most u, half a step of [1, 2). Of those there are 10 in the label's 32 columns (a chain of 8, and 2 that join four
    # chains), 4 between the parts of a tile's columns, and 2 roundings for each of the 4 parts of 300 words and their
    # joining: 32 at most. (A difference lse - logit would be off by u x, 71 u, for the largest rows, whose loss is 1e-28.)
    assert bool(((losses.double() - want).abs() <= 32 * vocab.U + want * (2.0 ** -20 + 16 * vocab.U * x)).all())
    assert not losses[16:].any()
    dh, dw = tr.linear_cross_entropy_backward(hidden, weight, labels, lse)
    want_h, want_w = vocab.linear_cross_entropy_backward(hidden, weight, labels, lse)
    close(dh, want_h)
    close(dw, want_w)


PART_STEPS = 64  # the logits are summed in parts of 1024 of the depth, a part in steps of 16


@pytest.mark.parametrize("rows,v", [(256, 5003), (600, 40)])
def test_small_calls_have_finer_sums(rows, v):
    """The logits of few tiles are summed in parts of 512, 32 steps. Each step rounds toward zero, by less than 2^-23 of a
    positive sum that is at most its part: 32 2^-23, 3.8e-6. The 3 additions of 2048 / 512 parts round to nearest, by u of the sum at most, with
    no side: over n rows their mean is below 3 u sqrt(57 / n) but once in 10^12. Scaling and adding the logarithm are two
    roundings, log2(e) and ln 2 are off by 2^-26. (Parts of 1024 are 5.4e-6 too small on average.)"""
    cols, g = 2048, gen(31)
    hidden = (0.5 + torch.rand(rows, cols, generator=g, device=DEV)).half()
    weight = torch.zeros(v, cols, device=DEV, dtype=torch.float16)
    weight[3] = (30.0 / cols * (0.5 + torch.rand(cols, generator=g, device=DEV))).half()
    labels = torch.full((rows,), 3, device=DEV)
    z = hidden.double() @ weight[3].double()
    exact = z + torch.log1p((v - 1) * torch.exp(-z))
    _, lse = tr.linear_cross_entropy(hidden, weight, labels)
    off = float(((lse.double() - exact) / exact).mean())
    assert abs(off) <= 32 * 2.0 ** -23 + 3 * vocab.U * (57.0 / rows) ** 0.5 + 2 * vocab.U + 2.0 ** -25, off


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(40, 32768), (300, 16392), (20000, 4104)])
def test_certain_rows_of_long_sums(rows, cols, dtype):
    """The label's logit is a sum of many positive products, and the label has all of the probability but 1e-11.

    A step of a part rounds its sum toward zero, by less than 2^-23 of it, and the sum is at most the part's: the parts are
    off by PART_STEPS 2^-23 of themselves, their sum by a rounding (u) for each part more. That is e, 3e-4 for a logit of 30. One
    sum over the whole depth would be off by 2048 such steps (at half of the final sum on average: 1e-3 and more for a logit of 30). The
    gradient's logits are the forward pass's own, bit for bit, so with the lse of that pass dz does not have that error: what is left are
    the roundings of z, of lse, of their products with log2(e) and ln 2 and of 2^x: 8 u (|z| + |lse|) + 2^-20."""
    g, dt, v = gen(cols), DTYPES[dtype], 300
    hidden = (0.5 + torch.rand(rows, cols, generator=g, device=DEV)).to(dt)
    weight = torch.zeros(v, cols, device=DEV, dtype=dt)
    weight[3] = (30.0 / cols * (0.5 + torch.rand(cols, generator=g, device=DEV))).to(dt)
    labels = torch.full((rows,), 3, device=DEV)
    h, w = hidden.double(), weight[3].double()
    z = h @ w
    exact = z + torch.log1p((v - 1) * torch.exp(-z))
    e = (PART_STEPS * 2.0 ** -23 + cols / 1024 * vocab.U) * z
    rest = 8 * vocab.U * (z + exact) + 2.0 ** -20
    losses, lse = tr.linear_cross_entropy(hidden, weight, labels)
    assert bool(((lse.double() - exact).abs() <= e + rest).all())
    assert bool((losses.double() <= 2.0 ** -20).all())
    # dz rounded to the type (T, and 2^-25 of float16's 2^-14), then the outputs
    t, tiny = vocab.HALF_STEP[dt]
    for given, off in ((lse, rest), (exact.float(), e + rest)):
        dh, dw = tr.linear_cross_entropy_backward(hidden, weight, labels, given)
        dz = off * (1 + t) + tiny * 2.0 ** -14 + torch.exp(-z) * v  # what dz may be: it is nearly 0 itself
        assert bool((dw[3].double().abs() <= (dz @ h) * (1 + 2 * t) + tiny).all())
        assert bool((dh.double().abs() <= dz[:, None] * w * (1 + 2 * t) + tiny).all())


FINE = [(1, 1024, 124), (2, 64, 31), (1, 8, 2), (18, 5568, 4645), (37, 1537, 5003), (201, 320, 136), (300, 65, 200), (872, 448, 25), (256, 72, 700)]


@pytest.mark.parametrize("rows,cols,v", FINE)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_small_gradients_are_rounded_once(rows, cols, v, dtype):
    """Where the products are short, dz is taken in two terms of the type: it is off by the square of its half step, and what is left is the
    outputs' own rounding. (In float16 with its room for small numbers: 2^-25 of 2^14 as before.)"""
    hidden, weight, labels, dloss, dlse = loss_inputs(rows, cols, v, dtype, ignored=0.1 if rows > 100 else 0.0)
    _, lse = tr.linear_cross_entropy(hidden, weight, labels)
    dh, dw = tr.linear_cross_entropy_backward(hidden, weight, labels, lse, dloss, dlse)
    want_h, want_w = vocab.linear_cross_entropy_backward(hidden, weight, labels, lse, dloss, dlse, terms=2)
    close(dh, want_h)
    close(dw, want_w)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_the_weights_gradient_of_few_rows_is_rounded_once(dtype):
    """Few rows of a long vocabulary: the weight's gradient has two terms of dz, the hidden one's long sums have one. Either alone is the same."""
    rows, cols, v = 100, 264, 30011
    hidden, weight, labels, dloss, dlse = loss_inputs(rows, cols, v, dtype, ignored=0.1)
    _, lse, dh, dw = check_loss(hidden, weight, labels, dloss, dlse)
    close(dw, vocab.linear_cross_entropy_backward(hidden, weight, labels, lse, dloss, dlse, terms=2)[1])
    assert same(tr.linear_cross_entropy_backward(hidden, weight, labels, lse, dloss, dlse, want_dweight=False)[0], dh)
    assert same(tr.linear_cross_entropy_backward(hidden, weight, labels, lse, dloss, dlse, want_dhidden=False)[1], dw)


GRAD_STEPS = 512  # the gradients are summed in parts of at most 8192 of the depth, a part in steps of 16


def signed_error(got, want):
    """(mean of the signed relative errors, what it may be). A step of a part rounds its sum toward zero, by less than 2^-23 of it, and where one
    large term comes first the sum is about the final one all the way: GRAD_STEPS 2^-23, 6e-5. The roundings to float16, at most
    2^-11 each to either side, leave a mean of n of them off by more than 2^-11 sqrt(57 / n) once in 10^12 (Hoeffding's inequality). One sum
    over 8192 steps is 2.5e-4 too small."""
    off = float(((got.double() - want) / want).mean())
    return off, GRAD_STEPS * 2.0 ** -23 + 2.0 ** -11 * (57.0 / want.numel()) ** 0.5


def test_a_hidden_gradient_of_many_words():
    """Even probabilities, 2^-17 each, so that all of dz is exact; the label's word, one of the first, gives nearly all of the gradient."""
    rows, cols, v = 1024, 2560, 1 << 17
    g = gen(21)
    hidden = torch.zeros(rows, cols, device=DEV, dtype=torch.float16)
    weight = torch.empty(v, cols, device=DEV, dtype=torch.float16)
    for part in weight.split(1 << 14):
        u = torch.rand(part.shape, generator=g, device=DEV) - 0.5
        part.copy_(u + 0.5 * torch.sign(u))
    weight.masked_fill_(weight == 0, 0.5)
    labels = torch.arange(rows, device=DEV)
    lse = torch.full((rows,), float(torch.log(torch.tensor(float(v), dtype=torch.float64))), device=DEV)
    dh, _ = tr.linear_cross_entropy_backward(hidden, weight, labels, lse, want_dweight=False)
    want = weight.sum(0, dtype=torch.float64) / v - weight[:rows].double()
    off, most = signed_error(dh, want)
    assert abs(off) <= most, (off, most)


def test_a_weight_gradient_of_many_rows():
    """Logits of 0, so that all of dz is exact; the first row gives nearly all of the gradient, and is so large that the others' products do not end
    within the bits of the sum."""
    rows, cols, v = 1 << 17, 2048, 16
    g = gen(22)
    weight = torch.zeros(v, cols, device=DEV, dtype=torch.float16)
    hidden = torch.empty(rows, cols, device=DEV, dtype=torch.float16)
    for part in hidden.split(1 << 14):
        part.copy_(2.0 ** -12 * torch.randn(part.shape, generator=g, device=DEV))
    hidden[0] = (8 + 8 * torch.rand(cols, generator=g, device=DEV)).half()
    labels = torch.full((rows,), 5, device=DEV)
    labels[0] = 3
    lse = torch.full((rows,), float(torch.log(torch.tensor(float(v), dtype=torch.float64))), device=DEV)
    _, dw = tr.linear_cross_entropy_backward(hidden, weight, labels, lse, want_dhidden=False)
    first = hidden[0].double()
    want = (hidden.sum(0, dtype=torch.float64) / v).repeat(v, 1)
    want[3] -= first
    keep = torch.arange(v, device=DEV) != 5  # (the sums of that word are of all the other rows)
    off, most = signed_error(dw[keep], want[keep])
    assert abs(off) <= most, (off, most)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_not_finite(dtype):
    """A row that holds no numbers spoils its own loss, and the gradients it is part of, and no other row's."""
    rows, cols, v = 300, 72, 400
    hidden, weight, labels, dloss, dlse = loss_inputs(rows, cols, v, dtype)
    clean = check_loss(hidden, weight, labels, dloss, dlse)
    bad = hidden.clone()
    bad[17, 3] = float("nan")
    bad[201] = float("inf")
    losses, lse = tr.linear_cross_entropy(bad, weight, labels)
    assert not bool(torch.isfinite(losses[[17, 201]]).any())
    ok = torch.ones(rows, dtype=torch.bool, device=DEV)
    ok[[17, 201]] = False
    assert same(losses[ok], clean[0][ok]) and same(lse[ok], clean[1][ok])
    dh, dw = tr.linear_cross_entropy_backward(bad, weight, labels, lse, dloss, dlse)
    assert same(dh[ok], clean[2][ok]) and not bool(torch.isfinite(dh[17]).any())
    # a word of the vocabulary that cannot be: its logit is minus infinity, its probability 0
    hidden, weight, labels, dloss, dlse = loss_inputs(rows, cols, v, dtype, seed=2)
    hidden[:, 0] = 1.0
    labels = labels % 50
    impossible = weight.clone()
    impossible[60] = 0.0
    impossible[60, 0] = float("-inf")
    losses, lse = tr.linear_cross_entropy(hidden, impossible, labels)
    rest = torch.cat([weight[:60], weight[61:]])
    z, e = vocab.logits(hidden, rest, 1.0)
    want = torch.logsumexp(z, 1)
    err = e.amax(1) + 2.0 ** -20 + (64 + v / 64) * vocab.U + 8 * vocab.U * (z.abs().amax(1) + want.abs())
    close(lse, (want, err))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_coefficients_that_are_not_finite(dtype, bad):
    """A row whose gradient of the loss or of the lse overflowed spoils its own hidden gradient, and takes no digits from the others'."""
    rows, cols, v = 300, 72, 400
    hidden, weight, labels, dloss, dlse = loss_inputs(rows, cols, v, dtype)
    _, lse = tr.linear_cross_entropy(hidden, weight, labels)
    ok = torch.ones(rows, dtype=torch.bool, device=DEV)
    ok[[17, 201]] = False
    zero = torch.zeros((), device=DEV)
    want, err = vocab.linear_cross_entropy_backward(hidden, weight, labels, lse, torch.where(ok, dloss, zero), torch.where(ok, dlse, zero), terms=2)[0]
    dloss[17] = bad
    dlse[201] = bad
    dh, dw = tr.linear_cross_entropy_backward(hidden, weight, labels, lse, dloss, dlse)
    close(dh[ok], (want[ok], err[ok]))
    assert not bool(torch.isfinite(dh[~ok]).any())


def test_float16_keeps_small_probabilities():
    """Probabilities far below float16's smallest number, with coefficients of a mean: the hidden gradient is theirs."""
    rows, cols, v = 64, 64, 4096
    g = gen(4)
    hidden = torch.zeros(rows, cols, device=DEV, dtype=torch.float16)
    weight = randn(g, (v, cols), torch.float16)
    labels = torch.full((rows,), v + 1, device=DEV)  # no label: nothing but the probabilities, 1 / 4096 each
    dloss = torch.full((rows,), 2.0 ** -13, device=DEV)
    losses, lse = tr.linear_cross_entropy(hidden, weight, labels)
    dh, _ = tr.linear_cross_entropy_backward(hidden, weight, labels, lse, dloss, logit_scale=2.0 ** 12)
    # dz = 2^-13 / 4096: exact in the scaled type; the sum over the words is in binary32
    want = 2.0 ** -13 * weight.double().sum(0) * 2.0 ** 12 / v
    size = 2.0 ** -13 * weight.double().abs().sum(0) * 2.0 ** 12 / v
    err = (v * vocab.U + 2.0 ** -20 + 64 * vocab.U) * size
    close(dh, (want.expand(rows, -1), err.expand(rows, -1)))


def test_one_gradient_at_a_time():
    hidden, weight, labels, dloss, dlse = loss_inputs(300, 136, 500, "bf16", ignored=0.2)
    _, lse, dh, dw = check_loss(hidden, weight, labels, dloss, dlse)
    only, none = tr.linear_cross_entropy_backward(hidden, weight, labels, lse, dloss, dlse, want_dweight=False)
    assert none is None and same(only, dh)
    none, only = tr.linear_cross_entropy_backward(hidden, weight, labels, lse, dloss, dlse, want_dhidden=False)
    assert none is None and same(only, dw)
    with pytest.raises(tr.TrError):
        tr.linear_cross_entropy_backward(hidden, weight, labels, lse, want_dhidden=False, want_dweight=False)


def test_no_rows():
    hidden, weight, labels, dloss, _ = loss_inputs(4, 16, 50, "f16")
    losses, lse = tr.linear_cross_entropy(hidden[:0], weight, labels[:0])
    assert losses.shape == (0,) and lse.shape == (0,)
    dh, dw = tr.linear_cross_entropy_backward(hidden[:0], weight, labels[:0], lse, dweight=torch.full_like(weight, 3.0))
    assert dh.shape == (0, 16) and not dw.any()


def test_loss_arguments():
    hidden, weight, labels, dloss, _ = loss_inputs(4, 16, 50, "f16")
    with pytest.raises(tr.TrError):
        tr.linear_cross_entropy(hidden.float(), weight.float(), labels)
    with pytest.raises(TypeError):
        tr.linear_cross_entropy(hidden, weight.bfloat16(), labels)
    with pytest.raises(ValueError):
        tr.linear_cross_entropy(hidden, weight[:, :8].contiguous(), labels)
    with pytest.raises(ValueError):
        tr.linear_cross_entropy(hidden[:, ::2], weight, labels)
    with pytest.raises(TypeError):
        tr.linear_cross_entropy(hidden, weight, labels.int())
    with pytest.raises(ValueError):
        tr.linear_cross_entropy(hidden, weight, labels[:3])
    with pytest.raises(ValueError):
        tr.linear_cross_entropy_backward(hidden, weight, labels, torch.zeros(3, device=DEV))
    with pytest.raises(TypeError):
        tr.linear_cross_entropy_backward(hidden, weight, labels, torch.zeros(4, device=DEV), dloss.double())
    with pytest.raises(tr.TrError):
        tr.linear_cross_entropy(hidden, weight, labels, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(tr.TrError):
        tr.linear_cross_entropy(hidden, weight, labels, logit_scale=float("nan"))


def test_outputs_end_where_they_end():
    """What lies behind the last row of every output stays, also where tiles reach past it."""
    rows, cols, v = 70, 72, 130
    hidden, weight, labels, dloss, dlse = loss_inputs(rows, cols, v, "bf16", ignored=0.1)
    for offset in (0, 1, 16):
        flat = [torch.full((n + 512,), 7.0, device=DEV, dtype=t) for n, t in
                ((rows, torch.float32), (rows, torch.float32), (rows * cols, torch.bfloat16), (v * cols, torch.bfloat16))]
        at = slice(128 + offset, None)
        view = lambda f, *shape: f[at][:torch.Size(shape).numel()].view(shape)  # noqa: E731
        losses, lse = tr.linear_cross_entropy(hidden, weight, labels, out=view(flat[0], rows), lse_out=view(flat[1], rows))
        dh, dw = tr.linear_cross_entropy_backward(hidden, weight, labels, lse, dloss, dlse, dhidden=view(flat[2], rows, cols),
                                                  dweight=view(flat[3], v, cols))
        want_h, want_w = vocab.linear_cross_entropy_backward(hidden, weight, labels, lse, dloss, dlse)
        close(dh, want_h)
        close(dw, want_w)
        for f, n in zip(flat, (rows, rows, rows * cols, v * cols)):
            assert bool((f[:128 + offset] == 7).all()) and bool((f[128 + offset + n:] == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("cols", [72, 520])
def test_gradients_in_different_places(dtype, cols):
    """dhidden and dweight that start anywhere, each while the other starts on 16 bytes; the bits are the same."""
    rows, v = 700, 1300
    hidden, weight, labels, dloss, dlse = loss_inputs(rows, cols, v, dtype, ignored=0.1)
    _, lse, dh, dw = check_loss(hidden, weight, labels, dloss, dlse)
    for oh, ow in ((1, 0), (0, 1), (3, 5)):
        flat_h = torch.full((rows * cols + 16,), 7.0, device=DEV, dtype=hidden.dtype)
        flat_w = torch.full((v * cols + 16,), 7.0, device=DEV, dtype=hidden.dtype)
        view_h, view_w = flat_h[oh:oh + rows * cols].view(rows, cols), flat_w[ow:ow + v * cols].view(v, cols)
        tr.linear_cross_entropy_backward(hidden, weight, labels, lse, dloss, dlse, dhidden=view_h, dweight=view_w)
        assert same(view_h, dh) and same(view_w, dw)
        assert bool((flat_h[:oh] == 7).all()) and bool((flat_h[oh + rows * cols:] == 7).all())
        assert bool((flat_w[:ow] == 7).all()) and bool((flat_w[ow + v * cols:] == 7).all())


@pytest.mark.parametrize("rows,cols,v", [(37, 65, 700), (300, 72, 130), (1100, 136, 1000), (200, 64, 5003)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_nothing_is_taken_from_a_workspace(rows, cols, v, dtype):
    """Workspaces and outputs that hold no numbers before the call; one workspace for calls of several sizes."""
    hidden, weight, labels, dloss, dlse = loss_inputs(rows, cols, v, dtype, ignored=0.3)
    ids = torch.randint(-1, v, (rows,), generator=gen(3), device=DEV)
    want = check_loss(hidden, weight, labels, dloss, dlse)
    n = max(tr.linear_cross_entropy_workspace_bytes(rows, cols, v, b) for b in (False, True))
    ws = torch.empty(max(n, tr.embedding_backward_workspace_bytes(rows, cols)), dtype=torch.uint8, device=DEV)
    half = rows // 2
    few = check_loss(hidden[:half], weight, labels[:half], dloss[:half], dlse[:half])
    clean = torch.nan_to_num(hidden)
    table = tr.embedding_backward(clean, ids, v)
    for part, expected in ((slice(None), want), (slice(half), few), (slice(None), want)):
        ws.fill_(255)
        h, l = hidden[part], labels[part]
        out = torch.full((2, h.shape[0]), float("nan"), device=DEV)
        tr.linear_cross_entropy(h, weight, l, out=out[0], lse_out=out[1], workspace=ws)
        ws.fill_(255)
        dh, dw = torch.full_like(h, float("nan")), torch.full_like(weight, float("nan"))
        tr.linear_cross_entropy_backward(h, weight, l, out[1], dloss[part], dlse[part], dhidden=dh, dweight=dw, workspace=ws)
        assert all(same(a, b) for a, b in zip((out[0], out[1], dh, dw), expected))
        ws.fill_(255)
        assert same(tr.embedding_backward(clean, ids, v, workspace=ws), table)


def test_a_workspace_of_a_longer_batch():
    """512 rows, whose pieces of the vocabulary are longer than those of 768, in the workspace of 768."""
    rows, cols, v = 512, 512, 250_000
    hidden, weight, labels, dloss, dlse = loss_inputs(rows, cols, v, "bf16")
    losses, lse = tr.linear_cross_entropy(hidden, weight, labels)
    want = tr.linear_cross_entropy_backward(hidden, weight, labels, lse, dloss, dlse)
    n = tr.linear_cross_entropy_workspace_bytes(768, cols, v, True)
    ws = torch.full((n + 4096,), 77, dtype=torch.uint8, device=DEV)
    got = tr.linear_cross_entropy_backward(hidden, weight, labels, lse, dloss, dlse, workspace=ws[:n])
    assert all(same(a, b) for a, b in zip(got, want))
    assert bool((ws[n:] == 77).all())


def test_losses_alone():
    """Without an lse to write."""
    hidden, weight, labels, _, _ = loss_inputs(70, 64, 300, "f16", ignored=0.2)
    losses, _ = tr.linear_cross_entropy(hidden, weight, labels)
    n = tr.linear_cross_entropy_workspace_bytes(70, 64, 300)
    ws, out = torch.empty(n, dtype=torch.uint8, device=DEV), torch.empty(70, device=DEV)
    assert tr.load().tr_linear_cross_entropy(tr.TR_F16, hidden.data_ptr(), weight.data_ptr(), labels.data_ptr(), out.data_ptr(), None, 70, 64,
                                             300, 1.0, IGNORE, 0, ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream) == tr.TR_OK
    assert same(out, losses)


def test_tables_past_32_bits():
    """Tables of more than 2^31 elements (4.4 GB): the rows at their ends."""
    v, cols = 1_080_000, 2048
    g = gen(12)
    table = torch.empty(v, cols, device=DEV, dtype=torch.bfloat16)
    table[:2000].normal_(generator=g)
    table[-2000:].normal_(generator=g)
    ends = torch.cat([torch.arange(2000, device=DEV), torch.arange(v - 2000, v, device=DEV)])
    ids = ends[torch.randperm(4000, generator=g, device=DEV)]
    assert torch.equal(tr.embedding(ids, table), table[ids])
    dy = randn(g, (4000, cols), torch.bfloat16)
    table.fill_(float("nan"))
    tr.embedding_backward(dy, ids, dtable=table)
    assert torch.equal(table[ids], dy)
    middle = table[2000:-2000].view(torch.int16)  # zeros everywhere else
    assert not any(bool(part.any()) for part in middle.split(100_000))


@pytest.mark.parametrize("cols", [4096, 4095])
def test_weights_past_32_bits(cols):
    """A weight of more than 2^31 elements, the gradients of three rows of hidden: the loss, and dweight's rows at both ends."""
    rows, v = 3, 530_000
    g = gen(13)
    weight = torch.empty(v, cols, device=DEV, dtype=torch.bfloat16)
    for part in weight.split(50_000):
        part.copy_(torch.randn(part.shape, generator=g, device=DEV) * (1.5 / cols ** 0.5))
    hidden = randn(g, (rows, cols), torch.bfloat16)
    labels = torch.tensor([v - 1, 0, v // 2], device=DEV)
    losses, lse = tr.linear_cross_entropy(hidden, weight, labels)
    z, e = zip(*(vocab.logits(hidden, part, 1.0) for part in weight.split(50_000)))
    z, e = torch.cat(z, 1), torch.cat(e, 1)
    want = torch.logsumexp(z, 1)
    err = e.amax(1) + 2.0 ** -20 + (64 + v / 64) * vocab.U + 8 * vocab.U * (z.abs().amax(1) + want.abs())
    close(lse, (want, err))
    picked = z.gather(1, labels[:, None])[:, 0]
    close(losses, (want - picked, err + e.gather(1, labels[:, None])[:, 0] + 8 * vocab.U * picked.abs()))
    dh, dw = tr.linear_cross_entropy_backward(hidden, weight, labels, lse)
    p = torch.exp(z - lse.double()[:, None])
    p_err = p * (e + 8 * vocab.U * (z.abs() + lse.double().abs()[:, None]) + 2.0 ** -20) + 4 * vocab.U * p
    p[torch.arange(rows, device=DEV), labels] -= 1.0
    p_err = p_err + 2.0 ** -8 * (p.abs() + p_err)  # its rounding to bfloat16
    h = hidden.double()
    for at in (slice(0, 4000), slice(v // 2 - 10, v // 2 + 10), slice(v - 4000, v)):
        q, qe = p[:, at], p_err[:, at]
        close(dw[at], (q.T @ h, qe.T @ h.abs() + (rows + 8) * vocab.U * (q.abs().T @ h.abs())))
    want_h, size, err_h = 0.0, 0.0, 0.0
    for i, part in enumerate(weight.split(50_000)):
        at = slice(50_000 * i, 50_000 * i + part.shape[0])
        w = part.double()
        want_h, size, err_h = want_h + p[:, at] @ w, size + p[:, at].abs() @ w.abs(), err_h + p_err[:, at] @ w.abs()
    close(dh, (want_h, err_h + (v + 8) * vocab.U * size))


# ---- streams, graphs, threads ---------------------------------------------------------------

def test_other_streams():
    hidden, weight, labels, dloss, dlse = loss_inputs(500, 264, 900, "bf16")
    ids = torch.randint(0, 900, (500,), generator=gen(1), device=DEV)
    base = check_loss(hidden, weight, labels, dloss, dlse)
    grad = tr.embedding_backward(hidden, ids, 900)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    out = []
    for _ in range(3):
        for s in streams:
            losses, lse = tr.linear_cross_entropy(hidden, weight, labels, stream=s)
            dh, dw = tr.linear_cross_entropy_backward(hidden, weight, labels, lse, dloss, dlse, stream=s)
            out.append((losses, lse, dh, dw, tr.embedding_backward(hidden, ids, 900, stream=s), tr.embedding(ids, weight, stream=s)))
    torch.cuda.synchronize()
    for got in out:
        assert all(same(a, b) for a, b in zip(got, (*base, grad, weight[ids])))


def test_threads():
    hidden, weight, labels, dloss, dlse = loss_inputs(300, 72, 700, "f16", ignored=0.1)
    ids = torch.randint(0, 700, (300,), generator=gen(2), device=DEV)
    dy = randn(gen(2), (300, 72), torch.float16)
    want = (*check_loss(hidden, weight, labels, dloss, dlse), tr.embedding_backward(dy, ids, 700))
    torch.cuda.synchronize()
    wrong = []

    def work():
        s = torch.cuda.Stream()
        for _ in range(10):
            losses, lse = tr.linear_cross_entropy(hidden, weight, labels, stream=s)
            dh, dw = tr.linear_cross_entropy_backward(hidden, weight, labels, lse, dloss, dlse, stream=s)
            got = (losses, lse, dh, dw, tr.embedding_backward(dy, ids, 700, stream=s))
            s.synchronize()
            if not all(same(a, b) for a, b in zip(got, want)):
                wrong.append(1)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("rows,cols,v", [(16, 64, 5003), (16, 400, 700), (300, 65, 2100)])
def test_products_end_before_what_follows(rows, cols, v):
    """Products of fewer blocks than the ring has stages, of as many and of more, each followed at once by kernels that begin early and use the
    shared memory that the products had: all of the arrivals at a product's barriers come before it ends, so nothing of them is found there."""
    hidden, weight, labels, dloss, dlse = loss_inputs(rows, cols, v, "bf16")
    ids = torch.randint(0, v, (rows,), generator=gen(11), device=DEV)
    want = (*check_loss(hidden, weight, labels, dloss, dlse), tr.embedding_backward(hidden, ids, v))
    torch.cuda.synchronize()
    out = []
    for _ in range(100):
        losses, lse = tr.linear_cross_entropy(hidden, weight, labels)
        grads = tr.linear_cross_entropy_backward(hidden, weight, labels, lse, dloss, dlse)
        out.append((losses, lse, *grads, tr.embedding_backward(hidden, ids, v)))
    torch.cuda.synchronize()
    assert tr.tr_last_device_error() == tr.TR_OK
    for got in out:
        assert all(same(a, b) for a, b in zip(got, want))


def test_graphs():
    """Captured once, replayed on other data; two graphs with a workspace each."""
    a, b = (loss_inputs(400, 136, 600, "bf16", seed=s, ignored=0.2 * s) for s in (0, 1))
    ids = [torch.randint(-1, 600, (400,), generator=gen(s), device=DEV) for s in (5, 6)]
    hidden, weight, labels, dloss, dlse = (t.clone() for t in a)
    tok = ids[0].clone()

    def step():
        losses, lse = tr.linear_cross_entropy(hidden, weight, labels)
        dh, dw = tr.linear_cross_entropy_backward(hidden, weight, labels, lse, dloss, dlse)
        tr.embedding_backward(dh, tok, dtable=dw, accumulate=True)
        return losses, lse, dh, dw, tr.embedding(tok, weight, scale=2.0)

    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    for data, t in ((a, ids[0]), (b, ids[1]), (a, ids[0])):
        for dst, src in zip((hidden, weight, labels, dloss, dlse), data):
            dst.copy_(src)
        tok.copy_(t)
        want = step()
        for g, out in zip(graphs, outs):
            g.replay()
            torch.cuda.synchronize()
            assert all(same(x, y) for x, y in zip(out, want))


FIRST_CALLS = """
import torch
import fp32_row_reduction_gb300 as tr
g = torch.Generator("cuda")
g.manual_seed(1)
table = torch.randn(500, {cols}, generator=g, device="cuda").to(torch.bfloat16)
ids = torch.randint(0, 500, ({rows},), generator=g, device="cuda")
labels = torch.roll(ids, 1)
def step():
    x = tr.embedding(ids, table, scale=0.1)
    losses, lse = tr.linear_cross_entropy(x, table, labels)
    dx, dtable = tr.linear_cross_entropy_backward(x, table, labels, lse)
    return x, losses, lse, dx, dtable, tr.embedding_backward(dx, ids, 500)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):  # nothing of the library has run before
    out = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, step()))
assert tr.tr_last_device_error() == tr.TR_OK
print("as eager")
"""


@pytest.mark.parametrize("rows,cols", [(40, 64), (20000, 65)])
def test_first_calls_of_a_process_may_be_captured(rows, cols):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(rows=rows, cols=cols)], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "as eager" in r.stdout, r.stderr[-2000:]


# ---- a model's two ends together --------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_step_of_a_tied_model(dtype):
    """Embedding, a block norm, the loss; back through all of them into one tied table, whose gradient is clipped. Each
    stage is checked on what the stage before it gave."""
    dt, tokens, cols, v = DTYPES[dtype], 3 * 111, 264, 1003
    g = gen(9)
    table = randn(g, (v, cols), dt, 1.5 / cols ** 0.5)
    branch = randn(g, (tokens, cols), dt, 0.5)
    weight = (1 + 0.1 * torch.randn(cols, generator=g, device=DEV))
    ids = torch.randint(0, v, (3, 111), generator=g, device=DEV)
    ids[1, 80:] = -1
    labels = torch.cat([ids[:, 1:], torch.full((3, 1), IGNORE, device=DEV)], 1).reshape(-1)
    labels[labels < 0] = IGNORE
    x = tr.embedding(ids, table, scale=cols ** 0.5)
    close(x, vocab.embedding(ids, table, cols ** 0.5))
    y, h = tr.gated_residual_norm(x.view(tokens, cols), branch, weight=weight, post=False)
    losses, lse = tr.linear_cross_entropy(y, table, labels)
    close(losses, vocab.linear_cross_entropy(y, table, labels)[0])
    dloss = torch.full((tokens,), 1.0 / int((labels != IGNORE).sum()), device=DEV)
    dy, dtable = tr.linear_cross_entropy_backward(y, table, labels, lse, dloss)
    want_y, want_t = vocab.linear_cross_entropy_backward(y, table, labels, lse, dloss)
    close(dy, want_y)
    close(dtable, want_t)
    back = tr.gated_residual_norm_backward(h, branch, dy, weight=weight, post=False)
    of_loss = dtable.clone()
    tr.embedding_backward(back.dx.view(3, 111, cols), ids, dtable=dtable, scale=cols ** 0.5, accumulate=True)
    sums, err = vocab.embedding_backward(back.dx.view(3, 111, cols), ids, v, cols ** 0.5, of_loss)
    close(dtable, (sums, err))
    before = dtable.double()
    norm = tr.clip_global_norm([dtable, back.dweight], 1e-3)
    total = float((before ** 2).sum() + (back.dweight.double() / (1e-3 / (float(norm) + 1e-6))).pow(2).sum()) ** 0.5
    assert abs(float(norm) - total) <= 1e-5 * total
    close(dtable, (before * (1e-3 / (float(norm) + 1e-6)), 16 * vocab.U * before.abs()))


# ---- waits that give up ------------------------------------------------------------------------

@pytest.fixture
def hook():
    assert tr.tr_last_device_error() == tr.TR_OK
    yield tr.tr_debug_force_wait_timeout
    tr.tr_debug_force_wait_timeout(0)
    tr.tr_last_device_error()


@pytest.mark.parametrize("rows,cols,v", [(40, 72, 700), (900, 520, 5003), (300, 33, 999)])
def test_waits_that_give_up(hook, rows, cols, v):
    """An extra wait that nothing ends is reported and changes nothing. Waits for tiles that give up are reported, and what
    the call computes is no number; the next call is right again."""
    hidden, weight, labels, dloss, dlse = loss_inputs(rows, cols, v, "bf16", ignored=0.2)
    want = check_loss(hidden, weight, labels, dloss, dlse)
    counted = labels != IGNORE

    def both():
        losses, lse = tr.linear_cross_entropy(hidden, weight, labels)
        dh, dw = tr.linear_cross_entropy_backward(hidden, weight, labels, want[1], dloss, dlse)
        return losses, lse, dh, dw

    hook(1)
    got = both()
    assert tr.tr_last_device_error() == tr.TR_ERR_DEVICE_TIMEOUT
    assert all(same(a, b) for a, b in zip(got, want))
    hook(2)
    losses, lse, dh, dw = both()
    assert tr.tr_last_device_error() == tr.TR_ERR_DEVICE_TIMEOUT
    assert bool(torch.isnan(losses[counted]).all()) and bool(torch.isnan(lse[counted]).all())
    assert bool(torch.isnan(dh[counted]).all()) and bool(torch.isnan(dw).all())
    assert not losses[~counted].any() and not dh[~counted].any()
    hook(0)
    assert all(same(a, b) for a, b in zip(both(), want))
    assert tr.tr_last_device_error() == tr.TR_OK


def test_waits_that_give_up_in_parts(hook):
    """The same where the weight's gradient is summed in parts."""
    hidden, weight, labels, dloss, dlse = loss_inputs(8300, 40, 300, "bf16", ignored=0.0)
    losses, lse, dh, dw = check_loss(hidden, weight, labels, dloss, dlse)
    for mode in (1, 2, 0):
        hook(mode)
        got = tr.linear_cross_entropy_backward(hidden, weight, labels, lse, dloss, dlse)
        assert tr.tr_last_device_error() == (tr.TR_ERR_DEVICE_TIMEOUT if mode else tr.TR_OK)
        if mode == 2:
            assert all(bool(torch.isnan(t).all()) for t in got)
        else:
            assert same(got[0], dh) and same(got[1], dw)
