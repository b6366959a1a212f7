"""GPU parity of the gated residual norm and its backward against the float64 definition.

Every element has its own bound, from the roundings of the formulas' binary32 steps and of
the output's type (oracle/block.py derives them); gradients are also tested against
differences of the float64 definition, along random directions.
"""
import numpy as np
import pytest
import torch

import fp32_row_reduction_gb300 as tr
from oracle import block

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
#: (rows, cols, gate rows): one element, one row, odd and ragged widths, widths at and past each
#: kernel's limits, few long rows, many short ones; a gate per channel, per group, per row
SHAPES = [(1, 1, 0), (1, 4096, 1), (2, 2, 2), (3, 5, 3), (17, 257, 1), (37, 1537, 0), (40, 64, 8), (6, 2048, 3),
          (48, 5120, 0), (12, 6144, 4), (130, 1024, 1), (5, 8192, 1), (4, 8200, 2), (3, 16384, 1), (2, 20000, 1),
          (2, 16392, 2), (3, 40001, 3), (700, 128, 7), (1300, 96, 1300), (2500, 40, 5), (641, 1000, 0), (333, 2049, 9),
          (320, 512, 320), (160, 776, 80),
          # rows of clusters of 2, 4 and 8 CTAs, whole and ragged; rows read again for each pass
          (3, 8192, 1), (5, 12288, 0), (3, 32768, 3), (4, 30001, 2), (2, 70001, 1), (1, 131080, 1)]
MODES = [(True, True), (False, True), (True, False)]
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tr.load()


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def within(got, want, bound, dtype, what):
    want, bound = np.asarray(want), block.rounded(want, bound, dtype)
    err = np.abs(host(got).reshape(want.shape) - want)
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside the bound, worst {np.nanmax(err / bound):.3g} of it at "
                           f"{np.unravel_index(np.nanargmax(err / bound), want.shape)}")


def make(rows, cols, groups, dtype, kind, post, pre, seed=0, offset=0, mean=0.3, weights=True):
    """Inputs; `offset` elements off the start of their buffers."""
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    layer = kind == "layernorm"

    def matrix(scale, mu=0.0):
        t = torch.randn(rows * cols + offset, generator=g, device=DEV) * scale + mu
        return t.to(DTYPES[dtype])[offset:].view(rows, cols)

    def vector(want, scale, mu, shape):
        return torch.randn(shape, generator=g, device=DEV) * scale + mu if want else None

    return dict(x=matrix(1.5, mean), branch=matrix(0.7, -mean), h=matrix(2.0, mean), dy=matrix(1.0) if pre else None,
                dh=matrix(0.5), post_weight=vector(post and weights, 0.3, 1.0, cols),
                post_bias=vector(post and layer and weights, 0.3, 0.0, cols),
                gate=vector(groups, 0.5, 0.5, (groups, cols)), weight=vector(pre and weights, 0.3, 1.0, cols),
                bias=vector(pre and layer and weights, 0.3, 0.0, cols))


def args(d, *names):
    return {k: d[k] for k in names}


def check_forward(d, dtype, kind, post, pre, rs=1.0, bs=1.0, **more):
    y, h = tr.gated_residual_norm(d["x"], d["branch"], **args(d, "post_weight", "post_bias", "gate", "weight", "bias"),
                                  eps=EPS, kind=kind, post=post, pre=pre, residual_scale=rs, branch_scale=bs, **more)
    (wy, ey), (wh, eh) = block.forward(host(d["x"]), host(d["branch"]), host(d["post_weight"]), host(d["post_bias"]),
                                       host(d["gate"]), host(d["weight"]), host(d["bias"]), EPS, kind, post, pre, rs, bs)
    if h is not None:
        within(h, wh, eh, dtype, "h")
    assert (y is None) == (not pre)
    if pre:
        within(y, wy, ey, dtype, "y")
    return y, h


def run_backward(d, kind, post, pre, rs=1.0, bs=1.0, **more):
    return tr.gated_residual_norm_backward(d["h"], d["branch"], **args(d, "dy", "dh", "post_weight", "post_bias", "gate", "weight"),
                                           eps=EPS, kind=kind, post=post, pre=pre, residual_scale=rs, branch_scale=bs, **more)


def expected(d, kind, post, pre, rs=1.0, bs=1.0):
    return block.backward(host(d["h"]), host(d["branch"]), host(d["dy"]), host(d["dh"]), host(d["post_weight"]),
                          host(d["post_bias"]), host(d["gate"]), host(d["weight"]), EPS, kind, post, pre, rs, bs)


def check_backward(d, dtype, kind, post, pre, rs=1.0, bs=1.0, **more):
    got = run_backward(d, kind, post, pre, rs, bs, **more)
    want = expected(d, kind, post, pre, rs, bs)
    for k, v in got._asdict().items():
        assert (v is None) == (k not in want), k
        if v is not None:
            within(v, *want[k], dtype if k in ("dx", "dbranch") else "f32", k)
    return got


@pytest.mark.parametrize("rows,cols,groups", SHAPES)
@pytest.mark.parametrize("kind", ["rmsnorm", "layernorm"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_forward(rows, cols, groups, kind, dtype):
    for post, pre in MODES:
        check_forward(make(rows, cols, groups, dtype, kind, post, pre, seed=rows), dtype, kind, post, pre, 0.9, 1.1)


@pytest.mark.parametrize("rows,cols,groups", SHAPES)
@pytest.mark.parametrize("kind", ["rmsnorm", "layernorm"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_backward(rows, cols, groups, kind, dtype):
    for post, pre in MODES:
        check_backward(make(rows, cols, groups, dtype, kind, post, pre, seed=rows), dtype, kind, post, pre, 0.9, 1.1)


@pytest.mark.parametrize("rows,cols,groups", [(5, 520, 1), (7, 33, 7), (64, 4096, 2), (200, 2056, 0)])
@pytest.mark.parametrize("kind", ["rmsnorm", "layernorm"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_rows_off_their_alignment(rows, cols, groups, kind, dtype):
    for offset in (1, 4):
        d = make(rows, cols, groups, dtype, kind, True, True, seed=3, offset=offset)
        check_forward(d, dtype, kind, True, True)
        check_backward(d, dtype, kind, True, True)
    # one matrix off, the others on their boundary; parameters off theirs
    d = make(rows, cols, groups, dtype, kind, True, True, seed=4)
    d["branch"] = make(rows, cols, groups, dtype, kind, True, True, seed=5, offset=3)["branch"]
    check_forward(d, dtype, kind, True, True)
    check_backward(d, dtype, kind, True, True)
    d = make(rows, cols, groups, dtype, kind, True, True, seed=6)
    for k in ("weight", "post_weight", "gate"):
        if d[k] is not None:
            d[k] = torch.cat([d[k].new_zeros(1), d[k].reshape(-1)])[1:].view(d[k].shape)
    check_forward(d, dtype, kind, True, True)
    check_backward(d, dtype, kind, True, True)


@pytest.mark.parametrize("rows,cols", [(4, 640), (3, 129), (2, 20001)])
@pytest.mark.parametrize("kind", ["rmsnorm", "layernorm"])
def test_absent_parts(rows, cols, kind):
    d = make(rows, cols, 0, "f32", kind, True, True, weights=False)  # no weights, biases or gate
    check_forward(d, "f32", kind, True, True)
    y, h = check_forward(d, "f32", kind, True, True, want_h=False)
    assert h is None
    check_backward(d, "f32", kind, True, True)
    d["dh"] = None  # the residual stream ends here
    check_backward(d, "f32", kind, True, True)
    g = run_backward(d, kind, True, True, want_params=False)
    want = expected(d, kind, True, True)
    assert all(v is None for k, v in g._asdict().items() if k not in ("dx", "dbranch"))
    within(g.dx, *want["dx"], "f32", "dx")
    within(g.dbranch, *want["dbranch"], "f32", "dbranch")


@pytest.mark.parametrize("wanted", ["dpost_w", "dpost_b", "dgate", "dpre_w", "dpre_b"])
@pytest.mark.parametrize("groups", [1, 3, 12])
def test_single_column_gradients(wanted, groups):
    """The C entry takes any subset of the column gradients."""
    rows, cols = 12, 264
    d = make(rows, cols, groups, "f32", "layernorm", True, True)
    out = torch.full((groups if wanted == "dgate" else 1, cols), 7.0, device=DEV)
    dx, da = torch.empty_like(d["h"]), torch.empty_like(d["h"])
    n = tr.gated_residual_norm_backward_workspace_bytes(rows, cols, "layernorm")
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    p = {k: out.data_ptr() if k == wanted else None for k in ("dpost_w", "dpost_b", "dgate", "dpre_w", "dpre_b")}
    st = tr.load().tr_gated_residual_norm_backward(
        1, 0, 3, d["h"].data_ptr(), d["branch"].data_ptr(), d["dy"].data_ptr(), d["dh"].data_ptr(), d["post_weight"].data_ptr(),
        d["post_bias"].data_ptr(), d["gate"].data_ptr(), groups, d["weight"].data_ptr(), dx.data_ptr(), da.data_ptr(),
        *p.values(), rows, cols, 1.0, 1.0, EPS, 0, ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    assert st == tr.TR_OK
    name = dict(dpost_w="dpost_weight", dpost_b="dpost_bias", dgate="dgate", dpre_w="dweight", dpre_b="dbias")[wanted]
    want = expected(d, "layernorm", True, True)[name]
    within(out if wanted == "dgate" else out[0], *want, "f32", name)


@pytest.mark.parametrize("kind", ["rmsnorm", "layernorm"])
def test_unneeded_inputs_may_be_absent(kind):
    d = make(6, 320, 2, "bf16", kind, True, False)
    g = tr.gated_residual_norm_backward(None, d["branch"], None, d["dh"], d["post_weight"], d["post_bias"], d["gate"], eps=EPS,
                                        kind=kind, pre=False)
    want = expected(d, kind, True, False)
    for k, v in g._asdict().items():
        if v is not None:
            within(v, *want[k], "bf16" if k in ("dx", "dbranch") else "f32", k)


@pytest.mark.parametrize("rows,cols", [(3, 512), (3, 515), (2, 30000)])
@pytest.mark.parametrize("kind", ["rmsnorm", "layernorm"])
def test_rows_far_from_zero_and_rows_of_zeros(rows, cols, kind):
    d = make(rows, cols, 1, "f32", kind, True, True, mean=1000.0)
    check_forward(d, "f32", kind, True, True)
    check_backward(d, "f32", kind, True, True)
    for k in ("x", "branch", "h"):
        d[k][-1] = 0.0
    check_forward(d, "f32", kind, True, True)
    check_backward(d, "f32", kind, True, True)


@pytest.mark.parametrize("cols", [768, 771, 17000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_row_spoils_no_other(cols, bad):
    d = make(9, cols, 3, "f32", "layernorm", True, True)
    y0, h0 = check_forward(d, "f32", "layernorm", True, True)
    g0 = run_backward(d, "layernorm", True, True)
    for k in ("x", "branch", "h"):
        d[k] = d[k].clone()
        d[k][4, 5] = bad
    y, h = tr.gated_residual_norm(d["x"], d["branch"], **args(d, "post_weight", "post_bias", "gate", "weight", "bias"), eps=EPS, kind="layernorm")
    g = run_backward(d, "layernorm", True, True)
    keep = torch.arange(9, device=DEV) != 4
    for a, b in ((y, y0), (h, h0), (g.dx, g0.dx), (g.dbranch, g0.dbranch)):
        assert torch.equal(a[keep], b[keep])
    assert torch.isnan(y[4]).all() and torch.isnan(g.dx[4]).all()
    assert torch.equal(g.dgate[[0, 2]], g0.dgate[[0, 2]])  # the other groups' gates


@pytest.mark.parametrize("cols", [4096, 4100, 777, 20000, 70000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layernorm_of_rows_whose_start_is_unlike_the_rest(cols, dtype):
    """The sums are taken about the mean of a row's first 32 elements. With all of the spread in those, the variance
    loses a factor of at most 1 + cols / 32 (the shift's squared distance from the mean is at most cols / 32 variances)."""
    d = make(6, cols, 1, dtype, "layernorm", True, True, seed=8, mean=0.0)
    for k in ("x", "branch", "h"):
        d[k][:, :32] += 64.0
    room = 1 + cols / 32
    y, h = tr.gated_residual_norm(d["x"], d["branch"], **args(d, "post_weight", "post_bias", "gate", "weight", "bias"), eps=EPS, kind="layernorm")
    (wy, ey), (wh, eh) = block.forward(host(d["x"]), host(d["branch"]), host(d["post_weight"]), host(d["post_bias"]),
                                       host(d["gate"]), host(d["weight"]), host(d["bias"]), EPS, "layernorm", True, True, 1.0, 1.0)
    within(h, wh, room * eh, dtype, "h")
    within(y, wy, room * ey, dtype, "y")
    got, want = run_backward(d, "layernorm", True, True), expected(d, "layernorm", True, True)
    for k, v in got._asdict().items():
        within(v, want[k][0], room * want[k][1], dtype if k in ("dx", "dbranch") else "f32", k)


@pytest.mark.parametrize("cols", [1, 31, 64, 4096, 4099, 9000])
def test_layernorm_of_constant_rows(cols):
    """No variance: the unit is exactly zero, so h is x + gate b_post and y is the bias, each rounded once."""
    x = torch.full((3, cols), 1234.5, device=DEV)
    b = torch.randn(cols, device=DEV)
    y, h = tr.gated_residual_norm(torch.zeros_like(x), x, None, None, None, None, b, kind="layernorm")
    assert torch.equal(h, torch.zeros_like(x)) and torch.equal(y, b.expand(3, cols))
    y, h = tr.gated_residual_norm(x, x, None, None, None, None, b, kind="layernorm")
    assert torch.equal(h, x) and torch.equal(y, b.expand(3, cols))


def test_many_rows_that_are_read_again():
    """More rows than clusters are worth: a CTA to a row."""
    d = make(160, 66001, 4, "bf16", "layernorm", True, True, seed=2)
    check_forward(d, "bf16", "layernorm", True, True)
    check_backward(d, "bf16", "layernorm", True, True)


def test_no_rows():
    d = make(0, 64, 2, "bf16", "layernorm", True, True)
    y, h = tr.gated_residual_norm(d["x"], d["branch"], **args(d, "post_weight", "post_bias", "gate", "weight", "bias"), kind="layernorm")
    assert y.shape == h.shape == (0, 64)
    for v in run_backward(d, "layernorm", True, True)[2:]:
        assert torch.equal(v, torch.zeros_like(v))


@pytest.mark.parametrize("rows,cols,groups", [(700, 1024, 1), (640, 515, 64), (300, 2048, 300), (5, 9000, 1),
                                              (400, 16384, 4), (90, 12289, 0), (7, 70000, 1)])
def test_results_repeat(rows, cols, groups):
    d = make(rows, cols, groups, "bf16", "layernorm", True, True)
    first = run_backward(d, "layernorm", True, True)
    for _ in range(3):
        for a, b in zip(run_backward(d, "layernorm", True, True), first):
            assert (a is None and b is None) or torch.equal(a, b)  # (no gate: no gradient of it)


@pytest.mark.parametrize("rows,cols", [(2, 4096), (300, 2560), (40, 1023), (3, 20000), (2, 70000)])
def test_captured_calls_follow_their_inputs(rows, cols):
    """Both directions in one graph, replayed on other inputs, beside an eager call on another stream."""
    d = make(rows, cols, 1, "bf16", "rmsnorm", True, True)
    other = make(rows, cols, 1, "bf16", "rmsnorm", True, True, seed=9)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = tr.gated_residual_norm(d["x"], d["branch"], **args(d, "post_weight", "gate", "weight"), eps=EPS)
        g = run_backward(d, "rmsnorm", True, True)
    for src in (other, make(rows, cols, 1, "bf16", "rmsnorm", True, True, seed=10)):
        for k, v in d.items():
            if v is not None:
                v.copy_(src[k])
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        g2 = run_backward(src, "rmsnorm", True, True, stream=side)  # at the same time, its own workspace
        y2, h2 = tr.gated_residual_norm(src["x"], src["branch"], **args(src, "post_weight", "gate", "weight"), eps=EPS, stream=side)
        torch.cuda.synchronize()
        for a, b in ((y, y2), (h, h2), *zip(g, g2)):
            assert a is None and b is None or torch.equal(a, b)
        check_forward(d, "bf16", "rmsnorm", True, True)


def test_outputs_go_where_they_are_asked():
    d = make(5, 264, 0, "f16", "rmsnorm", True, True)
    buf = torch.full((9, 264), 3.0, dtype=torch.float16, device=DEV)
    out, h_out = buf[2:7], torch.empty_like(d["x"])
    y, h = tr.gated_residual_norm(d["x"], d["branch"], out=out, h_out=h_out)
    assert y is out and h is h_out
    assert (buf[:2] == 3).all() and (buf[7:] == 3).all()
    dx = torch.full((9, 264), 3.0, dtype=torch.float16, device=DEV)
    g = run_backward(d, "rmsnorm", True, True, dx=dx[2:7])
    assert (dx[:2] == 3).all() and (dx[7:] == 3).all() and g.dx.data_ptr() == dx[2:7].data_ptr()


def test_refused_tensors():
    d = make(4, 64, 0, "bf16", "rmsnorm", True, True)
    f = tr.gated_residual_norm
    with pytest.raises(TypeError):
        f(d["x"], d["branch"].float())
    with pytest.raises(ValueError):
        f(d["x"], d["branch"][:3])
    with pytest.raises(ValueError):
        f(d["x"].t(), d["branch"].t())
    with pytest.raises(TypeError):
        f(d["x"], d["branch"], weight=d["weight"].bfloat16())
    with pytest.raises(ValueError):
        f(d["x"], d["branch"], weight=d["weight"][:32])
    with pytest.raises(TypeError):
        f(d["x"].double(), d["branch"].double())
    with pytest.raises(tr.TrError):
        f(d["x"], d["branch"], gate=torch.ones(3, 64, device=DEV))
    with pytest.raises(tr.TrError):
        f(d["x"], d["branch"], out=d["x"])
    with pytest.raises(tr.TrError):
        f(d["x"], d["branch"], order="ordered")
    with pytest.raises(tr.TrError):
        f(d["x"], d["branch"], bias=d["weight"])
    with pytest.raises(tr.TrError):
        run_backward(d, "rmsnorm", True, True, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(TypeError):
        run_backward(d, "rmsnorm", True, True, dx=torch.empty(4, 64, device=DEV))


@pytest.mark.parametrize("kind", ["rmsnorm", "layernorm"])
@pytest.mark.parametrize("cols", [96, 129])
def test_gradients_against_differences(kind, cols):
    """Along a random direction v: <gradient, v> against the central difference of the float64
    definition, step 1e-5. The kernel may be off by its elements' bounds times |v|; the difference
    by 1e-7 of the terms (as in the definitions' own test)."""
    rows, groups, step, layer = 12, 4, 1e-5, kind == "layernorm"
    d = make(rows, cols, groups, "f32", kind, True, True, seed=5)
    p = dict(x=host(d["x"]), a=host(d["branch"]), post_w=host(d["post_weight"]), post_b=host(d["post_bias"]),
             gate=host(d["gate"]), pre_w=host(d["weight"]), pre_b=host(d["bias"]))
    tail = dict(eps=EPS, kind=kind, post=True, pre=True, rs=0.8, bs=1.2)
    dy, dh = host(d["dy"]), host(d["dh"])

    def loss(**k):
        (y, _), (h, _) = block.forward(**{**p, **k}, **tail)
        return (y * dy).sum() + (h * dh).sum()

    h64 = block.forward(**p, **tail)[1][0]
    d["h"] = torch.from_numpy(h64).float().to(DEV)
    got = run_backward(d, kind, True, True, 0.8, 1.2)
    want = expected(d, kind, True, True, 0.8, 1.2)
    rng = np.random.default_rng(1)
    names = dict(x="dx", a="dbranch", post_w="dpost_weight", gate="dgate", pre_w="dweight")
    if layer:
        names.update(post_b="dpost_bias", pre_b="dbias")
    # h is rounded to binary32 here: its gradients move by that times the second derivatives, of order
    # one in these units, so 1e-6 of the terms is added for it
    for k, name in names.items():
        v = rng.normal(size=p[k].shape)
        slope = (loss(**{k: p[k] + step * v}) - loss(**{k: p[k] - step * v})) / (2 * step)
        g = host(getattr(got, name)).reshape(p[k].shape)
        room = (block.rounded(*want[name], "f32").reshape(p[k].shape) * np.abs(v)).sum()
        assert abs((g * v).sum() - slope) <= room + 1.1e-6 * (10 + np.abs(g * v).sum()), name


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows, and rows on both sides of the limit."""
    rows, cols = 32790, 65536
    g = torch.Generator(DEV)
    g.manual_seed(1)
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    a = torch.empty_like(x).normal_(generator=g)
    w = torch.rand(cols, generator=g, device=DEV) + 0.5
    y, h = tr.gated_residual_norm(x, a, w, None, w, w)
    pick = torch.tensor([0, 16383, 16384, 32767, 32768, rows - 1], device=DEV)
    d = dict(x=x[pick], branch=a[pick], post_weight=w, post_bias=None, gate=w.view(1, -1), weight=w, bias=None)
    (wy, ey), (wh, eh) = block.forward(host(d["x"]), host(d["branch"]), host(w), None, host(w), host(w), None, EPS, "rmsnorm", True, True, 1.0, 1.0)
    within(y[pick], wy, ey, "bf16", "y")
    within(h[pick], wh, eh, "bf16", "h")
    del y
    grads = tr.gated_residual_norm_backward(h, a, x, None, w, None, w, w, want_params=False, dx=torch.empty_like(x))
    sub = dict(h=h[pick], branch=a[pick], dy=x[pick], dh=None, post_weight=w, post_bias=None, gate=w.view(1, -1), weight=w)
    want = expected(sub, "rmsnorm", True, True)
    within(grads.dx[pick], *want["dx"], "bf16", "dx")
    within(grads.dbranch[pick], *want["dbranch"], "bf16", "dbranch")


FIRST_CALLS = """
import torch
import fp32_row_reduction_gb300 as tr
x = torch.randn(6, {cols}, device="cuda").to(torch.bfloat16)
w = torch.rand({cols}, device="cuda")
grads = [torch.randn(n, device="cuda") for n in (5, 70000)]
outs = [torch.empty_like(t) for t in grads]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):  # nothing of the library has run before
    y, h = tr.gated_residual_norm(x, x, w, None, w, w)
    g = tr.gated_residual_norm_backward(h, x, y, x, w, None, w, w)
    n = tr.clip_global_norm(grads + [g.dweight], 1.0, out=outs + [torch.empty_like(g.dweight)])
graph.replay()
torch.cuda.synchronize()
y2, h2 = tr.gated_residual_norm(x, x, w, None, w, w)
g2 = tr.gated_residual_norm_backward(h2, x, y2, x, w, None, w, w)
n2 = tr.clip_global_norm(grads + [g2.dweight], 1.0, out=[torch.empty_like(t) for t in grads + [g2.dweight]])
assert torch.equal(y, y2) and torch.equal(h, h2) and torch.equal(n, n2)
assert all(a is None or torch.equal(a, b) for a, b in zip(g, g2))
assert tr.tr_last_device_error() == tr.TR_OK
print("as eager")
"""


@pytest.mark.parametrize("cols", [1024, 16384, 70000])
def test_first_calls_of_a_process_may_be_captured(cols):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(cols=cols)], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "as eager" in r.stdout, r.stderr[-2000:]


def test_calls_from_several_threads():
    """Four threads, each with its own stream and shape (clusters among them), many calls each."""
    import threading
    cases = [make(r, c, 1, "bf16", "layernorm", True, True, seed=r) for r, c in ((200, 1024), (9, 12288), (64, 515), (3, 40000))]
    want = [(tr.gated_residual_norm(d["x"], d["branch"], kind="layernorm"), run_backward(d, "layernorm", True, True)) for d in cases]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        d, stream = cases[i], torch.cuda.Stream()
        for _ in range(20):
            fwd = tr.gated_residual_norm(d["x"], d["branch"], kind="layernorm", stream=stream)
            back = run_backward(d, "layernorm", True, True, stream=stream)
            stream.synchronize()
            if not all(torch.equal(a, b) for a, b in zip((*fwd, *back), (*want[i][0], *want[i][1]))):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    assert tr.tr_last_device_error() == tr.TR_OK


@pytest.mark.parametrize("rows,cols", [(1, 131080), (3, 70001)])
@pytest.mark.parametrize("kind", ["rmsnorm", "layernorm"])
def test_clusters_that_start_while_the_device_is_full(rows, cols, kind):
    """A cluster's CTAs may begin one after another: the first sums of a row wait for all of them. Calls are queued behind
    and beside launches that hold every SM, so that their CTAs start as SMs come free."""
    d = make(rows, cols, 1, "f32", kind, True, True, seed=12)
    y0, h0 = check_forward(d, "f32", kind, True, True)
    g0 = check_backward(d, "f32", kind, True, True)
    full = make(4000, 4096, 0, "bf16", kind, True, True, seed=13)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(10):
        tr.gated_residual_norm(full["x"], full["branch"], kind=kind, stream=side)
        got.append((tr.gated_residual_norm(d["x"], d["branch"], **args(d, "post_weight", "post_bias", "gate", "weight", "bias"),
                                           eps=EPS, kind=kind), run_backward(d, kind, True, True)))
    torch.cuda.synchronize()
    for (y, h), g in got:
        assert torch.equal(y, y0) and torch.equal(h, h0)
        assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(g, g0))
    assert tr.tr_last_device_error() == tr.TR_OK


@pytest.mark.parametrize("rows,cols", [(6, 777), (700, 1032), (6, 4096), (6, 4100), (300, 4096), (5, 9000), (6, 20000), (3, 40001),
                                       (2, 70000), (170, 70001)])
@pytest.mark.parametrize("kind_of_start", ["4 sigma", "16 sigma", "most of the variance"])
def test_layernorm_keeps_its_precision_when_a_row_starts_unlike_the_rest(rows, cols, kind_of_start):
    """Rows whose first 32 elements are far from the mean keep the ordinary bounds, all results alike. So do
    ordinary rows between them, whose results are the same bits as with no such neighbour."""
    d = make(rows, cols, 1, "f32", "layernorm", True, True, seed=21, mean=0.2)
    plain = {k: None if v is None else v.clone() for k, v in d.items()}
    far = torch.arange(rows, device=DEV) % 3 != 1
    for k, sigma in (("x", 1.5), ("branch", 0.7), ("h", 2.0)):
        shift = {"4 sigma": 4 * sigma, "16 sigma": -16 * sigma, "most of the variance": 500.0}[kind_of_start]
        d[k][:, :32] += shift * far[:, None]
    y, h = check_forward(d, "f32", "layernorm", True, True, 0.9, 1.1)
    g = check_backward(d, "f32", "layernorm", True, True, 0.9, 1.1)
    y0, h0 = check_forward(plain, "f32", "layernorm", True, True, 0.9, 1.1)
    g0 = run_backward(plain, "layernorm", True, True, 0.9, 1.1)
    for a, b in ((y, y0), (h, h0), (g.dx, g0.dx), (g.dbranch, g0.dbranch)):
        assert torch.equal(a[~far], b[~far])


@pytest.mark.parametrize("cols", [512, 4100, 20000])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_layernorm_of_16_bit_rows_that_start_unlike_the_rest(cols, dtype):
    d = make(40, cols, 8, dtype, "layernorm", True, True, seed=22)
    for k in ("x", "branch", "h"):
        d[k][:, :32] += 100.0
    check_forward(d, dtype, "layernorm", True, True)
    check_backward(d, dtype, "layernorm", True, True)


@pytest.fixture
def hook():
    """The testing modes of the bounded waits, off again afterwards."""
    assert tr.tr_last_device_error() == tr.TR_OK
    yield lambda mode: tr.tr_debug_force_wait_timeout(mode)
    tr.tr_debug_force_wait_timeout(0)
    tr.tr_last_device_error()


#: rows of clusters of 2, 4 and 8 CTAs in both directions, aligned and odd; gate rows of one slab, and several to a slab
CLUSTERED = [(5, 12288, 1, "bf16"), (7, 12289, 7, "f16"), (4, 32768, 2, "bf16"), (3, 16384, 1, "f32"), (2, 32767, 1, "f32"),
             (120, 8712, 120, "f32")]


@pytest.mark.parametrize("rows,cols,groups,dtype", CLUSTERED)
@pytest.mark.parametrize("kind", ["rmsnorm", "layernorm"])
def test_clusters_that_give_up_say_so_and_recover(hook, rows, cols, groups, dtype, kind):
    """Mode 4: every wait for the other CTAs of a row gives up. The call is reported, and what is computed from the row
    sums is NaN; what is not comes out as before (dbias, the plain sum of dy), and so do the next calls, with nothing reset
    but the error word."""
    d = make(rows, cols, groups, dtype, kind, True, True, seed=17)
    fwd = lambda: tr.gated_residual_norm(  # noqa: E731
        d["x"], d["branch"], **args(d, "post_weight", "post_bias", "gate", "weight", "bias"), eps=EPS, kind=kind)
    y0, h0 = fwd()
    g0 = run_backward(d, kind, True, True)
    torch.cuda.synchronize()
    assert hook(4) == tr.TR_OK
    for _ in range(3):
        y, h = fwd()
        g = run_backward(d, kind, True, True)
    assert hook(0) == tr.TR_OK
    y1, h1 = fwd()
    g1 = run_backward(d, kind, True, True)
    torch.cuda.synchronize()
    for t in (y, h, g.dx, g.dbranch, g.dpost_weight, g.dpost_bias, g.dgate, g.dweight):
        assert t is None or torch.isnan(t).all()
    assert kind == "rmsnorm" or torch.equal(g.dbias, g0.dbias)
    assert tr.tr_last_device_error() == tr.TR_ERR_DEVICE_TIMEOUT
    assert tr.tr_last_device_error() == tr.TR_OK
    for a, b in ((y1, y0), (h1, h0), *zip(g1, g0)):
        assert a is None and b is None or torch.equal(a, b)


@pytest.mark.parametrize("rows,cols,groups,dtype", CLUSTERED)
@pytest.mark.parametrize("mode", [1, 2])
def test_clusters_wait_out_a_barrier_that_nothing_completes(hook, mode, rows, cols, groups, dtype):
    """Mode 1: one wait runs out after its limit and is reported; results stay correct. Mode 2 has nothing to expire here."""
    d = make(rows, cols, groups, dtype, "layernorm", True, True, seed=18)
    fwd = lambda: tr.gated_residual_norm(  # noqa: E731
        d["x"], d["branch"], **args(d, "post_weight", "post_bias", "gate", "weight", "bias"), eps=EPS, kind="layernorm")
    y0, h0 = fwd()
    g0 = run_backward(d, "layernorm", True, True)
    for call, want in ((fwd, (y0, h0)), (lambda: run_backward(d, "layernorm", True, True), g0)):
        torch.cuda.synchronize()
        assert hook(mode) == tr.TR_OK
        got = call()
        assert hook(0) == tr.TR_OK
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert a is None and b is None or torch.equal(a, b)
        assert tr.tr_last_device_error() == (tr.TR_ERR_DEVICE_TIMEOUT if mode == 1 else tr.TR_OK)


@pytest.mark.parametrize("cols", [1024, 1031, 70001])
def test_rows_without_such_waits_are_not_changed_by_the_hook(hook, cols):
    """Rows of one CTA, and rows that are read again (whose CTAs meet in cluster barriers)."""
    d = make(4, cols, 1, "f32", "layernorm", True, True, seed=19)
    want = run_backward(d, "layernorm", True, True)
    assert hook(7) == tr.TR_OK
    got = run_backward(d, "layernorm", True, True)
    check_forward(d, "f32", "layernorm", True, True)
    assert hook(0) == tr.TR_OK
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert tr.tr_last_device_error() == tr.TR_OK


FAILED_LAUNCH = """
import ctypes
import torch
import fp32_row_reduction_gb300 as tr
rt = ctypes.CDLL(next(l.split()[-1] for l in open("/proc/self/maps") if "libcudart.so" in l))
x = torch.randn(6, 1024, device="cuda")
ts = [x.reshape(-1)]
y, h = torch.empty_like(x), torch.empty_like(x)
norm, sums = torch.zeros((), device="cuda"), torch.zeros(1024, device="cuda")
want = tr.axis_reduce(x, 0)
ptr, num, code = (ctypes.c_uint64 * 1)(x.data_ptr()), (ctypes.c_int64 * 1)(x.numel()), (ctypes.c_int32 * 1)(0)
torch.cuda.synchronize()
L = tr.load()
calls = {
    "forward": lambda: L.tr_gated_residual_norm(0, 0, 3, x.data_ptr(), x.data_ptr(), None, None, None, 0, None, None, h.data_ptr(),
                                                y.data_ptr(), 6, 1024, 1.0, 1.0, 1e-5, 0, None),
    "backward": lambda: L.tr_gated_residual_norm_backward(0, 0, 3, x.data_ptr(), x.data_ptr(), x.data_ptr(), None, None, None, None,
                                                          0, None, y.data_ptr(), h.data_ptr(), None, None, None, None, None, 6, 1024,
                                                          1.0, 1.0, 1e-5, 0, None, 0, None),
    "clip": lambda: L.tr_clip_by_norm(ctypes.addressof(ptr), None, ctypes.addressof(num), ctypes.addressof(code), 1, norm.data_ptr(),
                                      1.0, 1e-6, None),
}
for name, call in calls.items():
    handle, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert rt.cudaStreamCreate(ctypes.byref(handle)) == 0 and rt.cudaStreamBeginCapture(handle, 0) == 0
    status = call()  # the default stream may not be used while a stream it waits for is captured: refused on the host
    assert rt.cudaStreamEndCapture(handle, ctypes.byref(graph)) != 0
    rt.cudaGetLastError()
    assert status == tr.TR_ERR_CUDA, (name, status)
    got = tr.axis_reduce(x, 0)  # (raises where it finds that error again)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
print("not again")
"""


def test_a_failed_launch_is_not_reported_again_by_the_next_call():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FAILED_LAUNCH], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "not again" in r.stdout, r.stderr[-2000:]
