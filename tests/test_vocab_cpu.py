"""The embedding and the linear cross entropy without a GPU: refusals, workspace sizes, and the formulas of
the float64 oracle against differences and automatic differentiation."""
import ctypes

import pytest
import torch

import fp32_row_reduction_gb300 as tr
from fp32_row_reduction_gb300 import build as trbuild
from oracle import vocab

MB = 1 << 20
P = [1 << 30, 2 << 30, 3 << 30, 4 << 30, 5 << 30, 6 << 30, 7 << 30, 8 << 30, 9 << 30]  # made-up addresses, never read
INVALID, UNSUPPORTED = tr.TR_ERR_INVALID_ARG, tr.TR_ERR_UNSUPPORTED
BIG = 1 << 28


@pytest.fixture(scope="module")
def lib():
    trbuild.build()
    return tr.load()


def embed(lib, dtype=tr.TR_BF16, table=P[0], ids=P[1], out=P[2], tokens=4, vocab=100, cols=64, scale=1.0):
    return lib.tr_embedding(dtype, table, ids, out, tokens, vocab, cols, scale, None)


def embed_grad(lib, dtype=tr.TR_BF16, grad=tr.TR_BF16, dy=P[0], ids=P[1], dtable=P[2], tokens=4, vocab=100, cols=64, scale=1.0,
               accumulate=0, order=0, ws=P[3], n=BIG):
    return lib.tr_embedding_backward(dtype, grad, dy, ids, dtable, tokens, vocab, cols, scale, accumulate, order, ws, n, None)


def loss(lib, dtype=tr.TR_BF16, hidden=P[0], weight=P[1], labels=P[2], losses=P[3], lse=P[4], rows=4, cols=64, vocab=100, scale=1.0,
         ignore=-100, order=0, ws=P[5], n=BIG):
    return lib.tr_linear_cross_entropy(dtype, hidden, weight, labels, losses, lse, rows, cols, vocab, scale, ignore, order, ws, n, None)


def loss_grad(lib, dtype=tr.TR_BF16, hidden=P[0], weight=P[1], labels=P[2], lse=P[3], dloss=P[4], dlse=P[5], dhidden=P[6], dweight=P[7],
              rows=4, cols=64, vocab=100, scale=1.0, ignore=-100, order=0, ws=P[8], n=BIG):
    return lib.tr_linear_cross_entropy_backward(dtype, hidden, weight, labels, lse, dloss, dlse, dhidden, dweight, rows, cols, vocab,
                                                scale, ignore, order, ws, n, None)


NAN, INF = float("nan"), float("inf")
REFUSED = [
    (embed, dict(dtype=3)), (embed, dict(tokens=-1)), (embed, dict(vocab=0)), (embed, dict(vocab=1 << 31)), (embed, dict(cols=0)),
    (embed, dict(cols=1 << 24)), (embed, dict(scale=NAN)), (embed, dict(scale=INF)), (embed, dict(table=None)), (embed, dict(ids=None)),
    (embed, dict(out=None)), (embed, dict(table=P[0] + 1)), (embed, dict(ids=P[1] + 4)), (embed, dict(out=P[2] + 1)),
    (embed, dict(out=P[0] + 100 * 128 - 2)), (embed, dict(out=P[1])), (embed, dict(tokens=1 << 31)),
    (embed_grad, dict(dtype=-1)), (embed_grad, dict(grad=tr.TR_F16)), (embed_grad, dict(dtype=tr.TR_F32)), (embed_grad, dict(order=9)),
    (embed_grad, dict(tokens=-1)), (embed_grad, dict(vocab=0)), (embed_grad, dict(cols=0)), (embed_grad, dict(scale=INF)),
    (embed_grad, dict(accumulate=2)), (embed_grad, dict(dtable=None)), (embed_grad, dict(dy=None)), (embed_grad, dict(ids=None)),
    (embed_grad, dict(ws=None)), (embed_grad, dict(n=64)), (embed_grad, dict(ws=P[3] + 8)), (embed_grad, dict(dtable=P[0])),
    (embed_grad, dict(ws=P[2] + 4096)), (embed_grad, dict(dtable=P[2] + 1)), (embed_grad, dict(grad=tr.TR_F32, dtable=P[2] + 2)),
    (loss, dict(dtype=7)), (loss, dict(order=-1)), (loss, dict(rows=-1)), (loss, dict(cols=0)), (loss, dict(cols=1 << 24)),
    (loss, dict(vocab=0)), (loss, dict(vocab=1 << 24)), (loss, dict(scale=NAN)), (loss, dict(hidden=None)), (loss, dict(weight=None)),
    (loss, dict(labels=None)), (loss, dict(losses=None)), (loss, dict(weight=P[1] + 8)), (loss, dict(hidden=P[0] + 1)),
    (loss, dict(weight=P[1] + 1, cols=63)), (loss, dict(labels=P[2] + 4)), (loss, dict(losses=P[3] + 2)), (loss, dict(lse=P[3])),
    (loss, dict(losses=P[0])), (loss, dict(ws=None)), (loss, dict(n=16)), (loss, dict(ws=P[5] + 8)), (loss, dict(ws=P[1] + 16)),
    (loss_grad, dict(dtype=7)), (loss_grad, dict(order=4)), (loss_grad, dict(rows=-1)), (loss_grad, dict(cols=0)),
    (loss_grad, dict(vocab=0)), (loss_grad, dict(scale=INF)), (loss_grad, dict(dhidden=None, dweight=None)), (loss_grad, dict(lse=None)),
    (loss_grad, dict(hidden=None)), (loss_grad, dict(weight=None)), (loss_grad, dict(labels=None)), (loss_grad, dict(weight=P[1] + 2)),
    (loss_grad, dict(dhidden=P[0])), (loss_grad, dict(dweight=P[1])), (loss_grad, dict(dweight=P[6] + 64)), (loss_grad, dict(ws=None)),
    (loss_grad, dict(n=1024)), (loss_grad, dict(ws=P[6])), (loss_grad, dict(dloss=P[4] + 1)), (loss_grad, dict(dlse=P[5] + 2)),
]


@pytest.mark.parametrize("call,change", REFUSED, ids=lambda v: v.__name__ if callable(v) else "-".join(f"{k}={x}" for k, x in v.items()))
def test_refused(lib, call, change):
    assert call(lib, **change) == INVALID
    assert tr.tr_last_error_message()


@pytest.mark.parametrize("call", [embed_grad, loss, loss_grad])
@pytest.mark.parametrize("order", [tr.TR_ORDER_ORDERED_TREE, tr.TR_ORDER_FOLD_LEFT, tr.TR_ORDER_FOLD_RIGHT])
def test_orders_not_offered(lib, call, order):
    assert call(lib, order=order) == UNSUPPORTED


@pytest.mark.parametrize("call", [loss, loss_grad])
def test_float32_products_not_offered(lib, call):
    assert call(lib, dtype=tr.TR_F32) == UNSUPPORTED
    assert "float32" in tr.tr_last_error_message()


def test_nothing_to_do(lib):
    assert embed(lib, tokens=0, table=None, ids=None, out=None) == tr.TR_OK
    assert embed_grad(lib, tokens=0, accumulate=1, dy=None, ids=None, ws=None, n=0) == tr.TR_OK
    assert loss(lib, rows=0, hidden=None, labels=None, losses=None, lse=None, ws=None, n=0) == tr.TR_OK
    assert loss_grad(lib, rows=0, hidden=None, labels=None, lse=None, dloss=None, dlse=None, dweight=None, ws=None, n=0) == tr.TR_OK


def test_workspace_bytes(lib):
    n = ctypes.c_size_t(0)
    assert lib.tr_embedding_backward_workspace_bytes(16384, 4096, None) == INVALID
    assert lib.tr_embedding_backward_workspace_bytes(-1, 4096, ctypes.byref(n)) == INVALID
    assert lib.tr_linear_cross_entropy_workspace_bytes(8, 8, 8, 2, ctypes.byref(n)) == INVALID
    assert lib.tr_linear_cross_entropy_workspace_bytes(8, 8, 8, 0, None) == INVALID
    assert lib.tr_linear_cross_entropy_workspace_bytes(8, 8, 1 << 24, 0, ctypes.byref(n)) == INVALID
    assert tr.embedding_backward_workspace_bytes(0, 64) == 0
    assert tr.linear_cross_entropy_workspace_bytes(0, 64, 100) == 0
    # a little of the batch's own size: the sorted tokens and an eighth of the rows as partial sums
    assert tr.embedding_backward_workspace_bytes(16384, 4096) < 16384 * 4096 * 2 * 0.2
    # the forward pass keeps the packed rows and little else, far from the logits' 1.6 GB
    assert tr.linear_cross_entropy_workspace_bytes(8192, 4096, 50257) < 120 * MB
    # the backward pass keeps a piece of the logits' gradient
    assert tr.linear_cross_entropy_workspace_bytes(8192, 4096, 50257, True) < 600 * MB
    assert tr.linear_cross_entropy_workspace_bytes(8192, 4096, 250000, True) < 600 * MB
    # a longer call never needs less
    sizes = [tr.linear_cross_entropy_workspace_bytes(r, 512, 5003, True) for r in (1, 255, 256, 257, 5000, 40000, 400000)]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("v", [16, 300, 5003, 30000, 50257, 131072, 250000, 1100000])
@pytest.mark.parametrize("cols", [64, 136, 512, 2561, 4096, 20000])
def test_a_workspace_for_the_longest_batch_is_one_for_all(lib, cols, v, backward):
    """Sizes never fall as rows grow, for every number of tiles of 256 rows up to 40000 and some beyond."""
    rows = [1, 255, *range(256, 40000, 256), *(256 * 3 ** k for k in range(5, 13)), *(256 * 3 ** k + 1 for k in range(5, 13)), (1 << 31) - 1024]
    rows.sort()
    sizes = [tr.linear_cross_entropy_workspace_bytes(r, cols, v, backward) for r in rows]
    assert sizes == sorted(sizes)


def test_tensors_that_are_refused(lib):
    ids = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(TypeError):
        tr.embedding(ids, torch.zeros(4, 8))
    with pytest.raises(TypeError):
        tr.embedding_backward(torch.zeros(3, 8), ids, 4)
    with pytest.raises(TypeError):
        tr.linear_cross_entropy(torch.zeros(3, 8), torch.zeros(4, 8), ids)
    with pytest.raises(TypeError):
        tr.linear_cross_entropy_backward(torch.zeros(3, 8), torch.zeros(4, 8), ids, torch.zeros(3))


# ---- the oracle's formulas ----------------------------------------------------------

def case(rows=6, cols=5, v=7, seed=0):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(rows, cols, generator=g, dtype=torch.float64).half()
    w = torch.randn(v, cols, generator=g, dtype=torch.float64).half()
    labels = torch.tensor([0, v - 1, -100, v, -3, 2])[:rows]
    return h, w, labels, torch.randn(rows, generator=g), torch.randn(rows, generator=g)


def objective(h, w, labels, dloss, dlse, scale):
    (losses, _), (lse, _) = vocab.linear_cross_entropy(h, w, labels, scale)
    return float((losses * dloss + lse * dlse).sum())


@pytest.mark.parametrize("scale", [1.0, -0.5])
def test_gradients_against_differences(scale):
    h, w, labels, dloss, dlse = case()
    (_, _), (lse, _) = vocab.linear_cross_entropy(h, w, labels, scale)
    (dh, _), (dw, _) = vocab.linear_cross_entropy_backward(h, w, labels, lse, dloss, dlse, scale)
    step = 1e-5
    # the oracle takes any floating type: differences in float64, their error is step^2 and 1e-16 / step
    for t, grad, other in ((h.double(), dh, lambda x: (x, w.double())), (w.double(), dw, lambda x: (h.double(), x))):
        for i in range(t.shape[0]):
            for j in range(t.shape[1]):
                up, down = t.clone(), t.clone()
                up[i, j] += step
                down[i, j] -= step
                diff = (objective(*other(up), labels, dloss, dlse, scale) - objective(*other(down), labels, dloss, dlse, scale)) / (2 * step)
                assert abs(diff - float(grad[i, j])) < 1e-7


def test_gradients_against_autograd():
    h, w, labels, dloss, dlse = case()
    hh, ww = h.double().requires_grad_(), w.double().requires_grad_()
    z = hh @ ww.T
    counted = (labels != -100).double()
    inside = (labels >= 0) & (labels < w.shape[0])
    picked = torch.where(inside, z.gather(1, torch.where(inside, labels, 0)[:, None])[:, 0], torch.zeros(6, dtype=torch.float64))
    lse = torch.logsumexp(z, 1)
    (((lse - picked) * dloss + lse * dlse) * counted).sum().backward()
    (dh, _), (dw, _) = vocab.linear_cross_entropy_backward(h, w, labels, lse.detach(), dloss, dlse)
    assert torch.allclose(dh, hh.grad, atol=1e-13) and torch.allclose(dw, ww.grad, atol=1e-13)


def test_embedding_against_autograd():
    g = torch.Generator().manual_seed(3)
    table = torch.randn(9, 4, generator=g, dtype=torch.float64).requires_grad_()
    ids = torch.tensor([[0, 8, 3], [3, 3, 5]])
    dy = torch.randn(2, 3, 4, generator=g, dtype=torch.float64)
    (torch.nn.functional.embedding(ids, table) * 0.5 * dy).sum().backward()
    got, _ = vocab.embedding_backward(dy, ids, 9, 0.5)
    assert torch.allclose(got, table.grad, atol=1e-14)
    outside, _ = vocab.embedding(torch.tensor([-1, 9, 2]), table.detach(), 2.0)
    assert not outside[:2].any() and torch.equal(outside[2], 2 * table.detach()[2])
