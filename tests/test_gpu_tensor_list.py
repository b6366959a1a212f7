"""GPU parity of the global norm and of clipping, against float64 sums of the same elements.

Bounds, with u = 2^-24: a tile's squares meet in at most 20 binary32 operations in one thread
and then in binary64, so the sum is off by 20 u, its root by 10 u, the rounded norm by 12 u of itself. The factor
min(1, max_norm / (norm + eps)) adds an addition, a division and the product: 16 u of each
element, then the rounding to its type. "max" is exact.
"""
import math

import numpy as np
import pytest
import torch

import fp32_row_reduction_gb300 as tr
from oracle import block

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
NAMES = {v: k for k, v in DTYPES.items()}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tr.load()


def tensors(sizes, dtypes, seed=0, scale=1.0, offset=0):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        dt = DTYPES[dtypes[i % len(dtypes)]]
        off = (offset * i) % 9
        out.append((torch.randn(n + off, generator=g, device=DEV) * scale).to(dt)[off:])
    return out


def norm64(ts, kind="l2"):
    flat = np.concatenate([np.zeros(1)] + [t.double().cpu().numpy().reshape(-1) for t in ts])
    return float(np.sqrt((flat * flat).sum())) if kind == "l2" else float(np.abs(flat).max())


def check_norm(got, want, kind="l2"):
    assert got.dtype == torch.float32 and got.numel() == 1
    assert abs(float(got) - want) <= (12 * U * want + 2.0 ** -149 if kind == "l2" else 0.0), (float(got), want)


def check_scaled(before, after, want_norm, max_norm, eps=1e-6):
    f = min(1.0, max_norm / (want_norm + eps)) if not math.isinf(max_norm) else 1.0
    for b, a in zip(before, after):
        assert a.dtype == b.dtype and a.shape == b.shape
        want = b.double().cpu().numpy() * f
        err = np.abs(a.double().cpu().numpy() - want)
        assert (err <= block.rounded(want, 16 * U * np.abs(want), NAMES[b.dtype])).all()


SIZES = [
    [1], [4096], [5, 0, 1, 7, 8, 9, 15, 16, 17, 63], [8192] * 3 + [8191, 8193, 1],
    [1 << 20, 3, (1 << 18) + 5], [100] * 64, [33] * 65, [77, 1000, 12345] * 120,
]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("dtypes", [["f32"], ["bf16"], ["f16"], ["bf16", "f32", "f16"]], ids="-".join)
@pytest.mark.parametrize("offset", [0, 1])
def test_norm_and_clip(sizes, dtypes, offset):
    ts = tensors(sizes, dtypes, seed=len(sizes), offset=offset)
    copies = [t.clone() for t in ts]
    for kind in ("l2", "max"):
        want = norm64(ts, kind)
        check_norm(tr.global_norm(ts, kind=kind), want, kind)
        # into other tensors, whose places within 16 bytes differ from the tensors' own
        outs = [torch.empty(t.numel() + 5, dtype=t.dtype, device=DEV)[5 - (i % 5):][:t.numel()] for i, t in enumerate(ts)]
        n = tr.clip_global_norm(ts, 0.5 * want, kind=kind, out=outs)
        check_norm(n, want, kind)
        check_scaled(copies, outs, want, 0.5 * want)
        assert all(torch.equal(a, b) for a, b in zip(ts, copies))
    # in place
    want = norm64(ts)
    check_norm(tr.clip_global_norm(ts, 0.25), want)
    check_scaled(copies, ts, want, 0.25)


def test_many_tensors_take_several_launches():
    ts = tensors([3 + i % 50 for i in range(2500)], ["f32", "bf16"], offset=1)
    copies = [t.clone() for t in ts]
    want = norm64(ts)
    check_norm(tr.global_norm(ts), want)
    check_norm(tr.global_norm(ts, kind="max"), norm64(ts, "max"), "max")
    check_norm(tr.clip_global_norm(ts, 1.0), want)
    check_scaled(copies, ts, want, 1.0)


def test_nothing_outside_the_tensors_is_written():
    buf = torch.full((5000,), 2.0, dtype=torch.bfloat16, device=DEV)
    spans = [(3, 40), (41, 1001), (1002, 1010), (2001, 4994)]
    tr.clip_global_norm([buf[a:b] for a, b in spans], 1.0)
    inside = torch.zeros(5000, dtype=torch.bool, device=DEV)
    for a, b in spans:
        inside[a:b] = True
    assert (buf[~inside] == 2.0).all() and (buf[inside] < 1.0).all()
    src = [torch.ones(n, dtype=torch.float16, device=DEV) for n in (7, 33, 4097)]
    flat = torch.full((4200,), 9.0, dtype=torch.float16, device=DEV)
    tr.clip_global_norm(src, 1.0, out=[flat[1:8], flat[11:44], flat[51:4148]])
    assert (flat[[0, 8, 9, 10, 44, 50, 4148, 4199]] == 9.0).all() and (flat[51:4148] < 1).all()


def test_unclipped_tensors_are_copied_exactly():
    ts = tensors([1000, 77], ["f32", "bf16"])
    outs = [torch.empty_like(t) for t in ts]
    for max_norm in (1e6, float("inf")):
        tr.clip_global_norm(ts, max_norm, out=outs)
        assert all(torch.equal(a, b) for a, b in zip(ts, outs))
    tr.clip_global_norm(ts, 0.0, out=outs)
    assert all((o == 0).all() for o in outs)


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e-15, 1e18, 1e25, 1e36])
def test_squares_outside_binary32(scale):
    ts = [t * scale for t in tensors([10000, 3], ["f32"])]
    want = norm64(ts)
    check_norm(tr.global_norm(ts), want)
    # large and small together
    ts += tensors([500, 20], ["bf16", "f16"], seed=3)
    check_norm(tr.global_norm(ts), norm64(ts))


def test_special_values():
    ts = tensors([100, 5000], ["f32"])
    zeros = [torch.zeros(300, device=DEV), torch.zeros(9, dtype=torch.bfloat16, device=DEV)]
    assert float(tr.global_norm(zeros)) == 0.0 and float(tr.global_norm(zeros, kind="max")) == 0.0
    outs = [torch.ones_like(t) for t in zeros]
    assert float(tr.clip_global_norm(zeros, 1.0, out=outs)) == 0.0
    assert all((o == 0).all() for o in outs)
    ts[1][4999] = float("inf")
    for kind in ("l2", "max"):
        assert math.isinf(float(tr.global_norm(ts, kind=kind)))
    outs = [torch.empty_like(t) for t in ts]
    tr.clip_global_norm(ts, 1.0, out=outs)
    assert (outs[0] == 0).all() and (outs[1][:4999] == 0).all() and torch.isnan(outs[1][4999])
    ts[0][3] = float("nan")
    for kind in ("l2", "max"):
        assert math.isnan(float(tr.global_norm(ts, kind=kind)))
    tr.clip_global_norm(ts, 1.0, out=outs)
    assert all(torch.isnan(o).all() for o in outs)


def test_empty_lists():
    assert float(tr.global_norm([])) == 0.0
    assert float(tr.clip_global_norm([], 1.0)) == 0.0
    e = torch.empty(0, device=DEV)
    assert float(tr.clip_global_norm([e, e], 1.0)) == 0.0
    tr.clip_by_norm([], torch.ones((), device=DEV), 1.0)


def test_dense_tensors_of_any_order_and_overlapping_reads():
    t = torch.randn(40, 50, 6, device=DEV)
    p = t.permute(2, 0, 1)
    check_norm(tr.global_norm([p, t, t]), math.sqrt(3) * norm64([t]))
    out = torch.empty_like(p)
    assert out.stride() == p.stride()
    tr.clip_global_norm([p], 1.0, out=[out])
    check_scaled([p], [out], norm64([t]), 1.0)
    with pytest.raises(ValueError):
        tr.global_norm([t[:, ::2]])
    with pytest.raises(ValueError):
        tr.clip_global_norm([p], 1.0, out=[p.contiguous()])
    with pytest.raises(tr.TrError):
        tr.clip_global_norm([t, t], 1.0)
    with pytest.raises(TypeError):
        tr.global_norm([t.double()])
    with pytest.raises(TypeError):
        tr.global_norm([t, t.cpu()])
    with pytest.raises(ValueError):
        tr.clip_global_norm([t], 1.0, out=[])


def test_clip_by_a_given_norm():
    ts = tensors([300, 70000, 5], ["bf16", "f32"], offset=1)
    copies = [t.clone() for t in ts]
    norm = torch.full((1,), 80.0, device=DEV)
    outs = [torch.empty_like(t) for t in ts]
    tr.clip_by_norm(ts, norm, 20.0, out=outs)
    check_scaled(copies, outs, 80.0, 20.0)
    tr.clip_by_norm(ts, norm, 20.0)
    check_scaled(copies, ts, 80.0, 20.0)
    # squares summed over parts of a list, as several processes would
    parts = [tr.global_norm(copies[:1]), tr.global_norm(copies[1:])]
    both = torch.stack([p * p for p in parts]).sum().sqrt()
    assert abs(float(both) - norm64(copies)) <= 20 * U * norm64(copies)


def test_results_repeat_and_graphs_follow_their_inputs():
    ts = tensors([100000, 33, 4096, 70001], ["bf16", "f32"])
    outs = [torch.empty_like(t) for t in ts]
    first = tr.global_norm(ts)
    assert all(torch.equal(tr.global_norm(ts), first) for _ in range(3))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = tr.clip_global_norm(ts, 1.0, out=outs)
    side = torch.cuda.Stream()
    for seed in (5, 6):
        new = tensors([100000, 33, 4096, 70001], ["bf16", "f32"], seed=seed)
        for t, n in zip(ts, new):
            t.copy_(n)
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        outs2 = [torch.empty_like(t) for t in new]
        norm2 = tr.clip_global_norm(new, 1.0, out=outs2, stream=side)  # at the same time, its own workspace
        torch.cuda.synchronize()
        assert torch.equal(norm, norm2) and all(torch.equal(a, b) for a, b in zip(outs, outs2))
        check_norm(norm, norm64(new))


def test_a_tensor_past_32_bits():
    """A tensor of more than 2^32 bytes and 2^31 elements."""
    n = (1 << 31) + 1000
    t = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    t[[0, 1 << 30, (1 << 31) - 1, 1 << 31, n - 1]] = torch.tensor([1.0, 2.0, 4.0, 8.0, 16.0], dtype=torch.bfloat16, device=DEV)
    check_norm(tr.global_norm([t]), math.sqrt(1 + 4 + 16 + 64 + 256))
    tr.clip_by_norm([t], torch.ones((), device=DEV), 0.5)
    assert t[[0, 1 << 30, (1 << 31) - 1, 1 << 31, n - 1]].tolist() == [0.5, 1.0, 2.0, 4.0, 8.0]


def test_a_training_step_of_two_blocks():
    """Forward and backward through two block ends (the second one's h is the first one's residual
    stream), then all parameter gradients clipped together, against float64 throughout.
    Tolerance: every value meets a few hundred binary32 roundings of terms its own size or of a
    row's, so 2e-5 of the largest magnitude of its tensor (300 u) holds with room."""
    rows, cols, groups = 96, 640, 4
    g = torch.Generator(DEV)
    g.manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, a1, a2, dy = r(rows, cols), r(rows, cols), r(rows, cols), r(rows, cols)
    p1 = dict(post_weight=1 + 0.1 * r(cols), gate=r(groups, cols), weight=1 + 0.1 * r(cols))
    p2 = dict(post_weight=1 + 0.1 * r(cols), gate=r(cols), weight=1 + 0.1 * r(cols))
    y1, h1 = tr.gated_residual_norm(x, a1, **p1)
    y2, h2 = tr.gated_residual_norm(h1, a2 + y1, **p2)  # the second branch adds the normed stream
    b2 = tr.gated_residual_norm_backward(h2, a2 + y1, dy, None, **p2)
    b1 = tr.gated_residual_norm_backward(h1, a1, b2.dbranch, b2.dx, **p1)
    grads = [b1.dpost_weight, b1.dgate, b1.dweight, b2.dpost_weight, b2.dgate, b2.dweight]
    before = [t.clone() for t in grads]
    norm = tr.clip_global_norm(grads, 1.0)
    torch.cuda.synchronize()

    leaves = {k: v.double().requires_grad_() for k, v in dict(x=x, a1=a1, a2=a2, **{k + "1": v for k, v in p1.items()}, **{k + "2": v for k, v in p2.items()}).items()}
    rms = lambda v, w: v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-5) * w  # noqa: E731
    L = leaves
    s1 = L["x"] + L["gate1"].repeat_interleave(rows // groups, 0) * rms(L["a1"], L["post_weight1"])
    z1 = rms(s1, L["weight1"])
    s2 = s1 + L["gate2"] * rms(L["a2"] + z1, L["post_weight2"])
    z2 = rms(s2, L["weight2"])
    names = ["post_weight1", "gate1", "weight1", "post_weight2", "gate2", "weight2", "x", "a1", "a2"]
    want = torch.autograd.grad(z2, [L[k] for k in names], dy.double())
    near = lambda got, ref: float((got.double() - ref).abs().max()) <= 2e-5 * float(ref.abs().max())  # noqa: E731
    assert near(y2, z2.detach()) and near(h2, s2.detach())
    for got, ref, k in zip(before + [b1.dx, b1.dbranch, b2.dbranch], want, names):
        assert near(got, ref.reshape(got.shape)), k
    total = math.sqrt(sum(float((w * w).sum()) for w in want[:6]))
    assert abs(float(norm) - total) <= 2e-5 * total
    for got, ref in zip(grads, want):
        assert near(got, ref.reshape(got.shape) / (total + 1e-6))
