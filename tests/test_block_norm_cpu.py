"""The block norms and the norms over lists without a GPU: refused arguments, empty
calls, and the float64 definitions the GPU tests compare with, against differences."""
import array
import ctypes
import os
import subprocess

import numpy as np
import pytest

import fp32_row_reduction_gb300 as tr
from fp32_row_reduction_gb300 import build as trbuild
from oracle import block

OK, E, U = tr.TR_OK, tr.TR_ERR_INVALID_ARG, tr.TR_ERR_UNSUPPORTED
BASE = 1 << 20  # host-side stand-ins for device addresses: nothing here reaches CUDA


@pytest.fixture(scope="module", autouse=True)
def lib():
    trbuild.build()
    return tr.load()


def at(k):
    return BASE + (k << 16)


def fwd(**k):
    v = dict(kind=0, dtype=0, norms=3, x=at(0), branch=at(1), post_w=None, post_b=None, gate=None, gate_rows=0, pre_w=None,
             pre_b=None, h=at(2), y=at(3), rows=4, cols=8, rs=1.0, bs=1.0, eps=1e-5, order=0)
    v.update(k)
    return tr.load().tr_gated_residual_norm(*v.values(), None)


def bwd(**k):
    v = dict(kind=0, dtype=0, norms=3, h=at(0), branch=at(1), dy=at(2), dh=None, post_w=None, post_b=None, gate=None,
             gate_rows=0, pre_w=None, dx=at(3), dbranch=at(4), dpost_w=None, dpost_b=None, dgate=None, dpre_w=None,
             dpre_b=None, rows=4, cols=8, rs=1.0, bs=1.0, eps=1e-5, order=0, ws=None, ws_bytes=0)
    v.update(k)
    return tr.load().tr_gated_residual_norm_backward(*v.values(), None)


COMMON = [
    (dict(kind=2), E), (dict(dtype=3), E), (dict(dtype=-1), E), (dict(norms=0), E), (dict(norms=4), E), (dict(norms=-1), E),
    (dict(order=7), E), (dict(order=1), U), (dict(order=2), U), (dict(order=3), U),
    (dict(rows=-1), E), (dict(cols=0), E), (dict(cols=1 << 24), E), (dict(rows=1 << 40, cols=(1 << 24) - 1), E),
    (dict(eps=-1.0), E), (dict(eps=float("nan")), E), (dict(eps=float("inf")), E),
    (dict(rs=float("inf")), E), (dict(bs=float("nan")), E),
    (dict(gate=at(6), gate_rows=0), E), (dict(gate=at(6), gate_rows=3), E), (dict(gate=at(6), gate_rows=8), E),
    (dict(gate=at(6), gate_rows=-4), E), (dict(gate=at(6) + 2, gate_rows=2), E),
    (dict(post_w=at(6) + 1), E), (dict(post_b=at(6)), E), (dict(norms=2, post_w=at(6)), E),
    (dict(norms=1, pre_w=at(6)), E), (dict(branch=at(1) + 2), E), (dict(branch=at(1) + 1, dtype=1), E),
]


@pytest.mark.parametrize("args,status", COMMON + [
    (dict(x=None), E), (dict(branch=None), E), (dict(y=None), E), (dict(norms=1), E), (dict(norms=1, y=None, h=None), E),
    (dict(pre_b=at(6)), E), (dict(h=at(0)), E), (dict(y=at(1) + 64), E), (dict(y=at(2)), E),
    (dict(gate=at(3), gate_rows=4), E), (dict(post_w=at(2) + 32), E),
])
def test_forward_refuses(args, status):
    assert fwd(**args) == status
    assert "gated residual norm" in tr.tr_last_error_message()


@pytest.mark.parametrize("args,status", COMMON + [
    (dict(dx=None), E), (dict(dbranch=None), E), (dict(dy=None), E), (dict(h=None), E), (dict(branch=None), E),
    (dict(norms=1, dy=None), E),                 # no upstream gradient at all
    (dict(norms=1, dh=at(5)), E),                # dy without a pre-norm
    (dict(norms=2, branch=None, gate=at(6), gate_rows=2, dgate=at(7), ws=at(8), ws_bytes=1 << 16), E),
    (dict(dpost_b=at(6), ws=at(8), ws_bytes=1 << 16), E), (dict(norms=2, dpost_w=at(6), ws=at(8), ws_bytes=1 << 16), E),
    (dict(norms=1, dy=None, dh=at(2), dpre_w=at(6), ws=at(8), ws_bytes=1 << 16), E),
    (dict(dgate=at(6), ws=at(8), ws_bytes=1 << 16), E),
    (dict(dpre_w=at(6)), E), (dict(dpre_w=at(6), ws=at(8), ws_bytes=64), E), (dict(dpre_w=at(6), ws=at(8) + 4, ws_bytes=1 << 16), E),
    (dict(dpre_w=at(6), ws=at(6), ws_bytes=1 << 16), E), (dict(dpre_w=at(6), ws=at(2), ws_bytes=1 << 16), E),
    (dict(dx=at(0)), E), (dict(dx=at(2)), E), (dict(dbranch=at(1)), E), (dict(dx=at(4)), E), (dict(dh=at(3) + 4), E),
])
def test_backward_refuses(args, status):
    assert bwd(**args) == status
    assert "gated residual norm backward" in tr.tr_last_error_message()


def test_no_rows_is_a_no_op():
    assert fwd(rows=0, x=None, branch=None, h=None, y=None) == OK
    assert fwd(rows=0, gate=at(6), gate_rows=3) == OK
    assert bwd(rows=0, dx=None, dbranch=None, h=None, branch=None, dy=None) == OK
    assert tr.gated_residual_norm_backward_workspace_bytes(0, 8) == 0


def test_workspace_sizes():
    b = tr.gated_residual_norm_backward_workspace_bytes
    assert b(1, 8) == 32 + 2 * 8 * 4
    assert b(1, 8, "layernorm") == 32 + 4 * 8 * 4
    assert b(10 ** 6, 4096) < 10 ** 6 * 32 + (16 << 20)
    assert b(5, (1 << 24) - 1) < 1 << 28  # long rows: few partials
    n = ctypes.c_size_t(0)
    f = tr.load().tr_gated_residual_norm_backward_workspace_bytes
    assert f(0, -1, 8, ctypes.byref(n)) == E and f(0, 1, 0, ctypes.byref(n)) == E and f(2, 1, 8, ctypes.byref(n)) == E
    assert f(0, 1, 8, None) == E


SHAPES_PROGRAM = r"""
#include <cstdio>
#include "tr_block_rows.cuh"
using namespace tr::block;
static int bad = 0;
#define CHECK(what) do { if (!(what) && bad++ < 20) std::printf("%s: T %d cols %d odd %d layer %d tensors %d\n", #what, static_cast<int>(sizeof(T)), cols, odd, layer, tensors); } while (0)
template <class T>
static void sweep() {
    bool seen[2][5][2] = {};  // direction, slots, cluster
    for (int cols = 1; cols < 140000; ++cols)
        for (int odd = cols * static_cast<int>(sizeof(T)) % 16 != 0; odd < 2; ++odd)
            for (int layer = 0; layer < 2; ++layer)
                for (int tensors = 2; tensors <= 4; ++tensors)
                    for (int back = 0; back < 2; ++back) {
                        if (!back && tensors > 2) continue;
                        int slots = 0;
                        const RowShape g = back ? row_shape<T>(cols, tensors, odd, layer, 4, sizeof(T) == 2 ? 64 : 0, kBwdColumns, &slots)
                                                : row_shape<T>(cols, tensors, odd, layer, layer ? 4 : 3, 0, kFwdColumns, &slots);
                        if (g.warps == 0) {
                            CHECK(cols > (back ? 32768 : 65536));
                            continue;
                        }
                        CHECK(cols <= (back ? 32768 : 65536));
                        CHECK(slots >= 1 && slots * 16 <= (back ? kBwdColumns : kFwdColumns) * static_cast<int>(sizeof(T)));
                        CHECK(g.cluster == 1 || cluster_slots<T>(slots, back ? kBwdColumns : kFwdColumns));
                        CHECK(g.cluster == 1 || g.teams == 1);
                        CHECK(g.teams * g.warps <= kMaxWarps && row_smem(g) <= 226 * 1024);
                        CHECK(static_cast<long>(g.warps) * 32 * slots >= g.cta_vecs);                       // the threads cover the slots
                        CHECK(static_cast<long>(g.cta_vecs) * g.cluster * 16 >= cols * static_cast<long>(sizeof(T)));  // the CTAs the row,
                        CHECK(static_cast<long>(g.cta_vecs) * (g.cluster - 1) * 16 < cols * static_cast<long>(sizeof(T)));  // and each has some
                        if (!back && sizeof(T) == 2 && slots == 1) CHECK(g.teams * g.warps <= 10);
                        seen[back][slots][g.cluster > 1] = true;
                    }
    // every kernel that is compiled is reached
    const int cols = 0, odd = 0, layer = 0, tensors = 0;
    for (int back = 0; back < 2; ++back)
        for (int slots = 1; slots * 16 <= (back ? kBwdColumns : kFwdColumns) * static_cast<int>(sizeof(T)); ++slots) {
            CHECK(seen[back][slots][0]);
            CHECK(seen[back][slots][1] == cluster_slots<T>(slots, back ? kBwdColumns : kFwdColumns));
        }
}
int main() {
    sweep<float>();
    sweep<__half>();
    return bad != 0;
}
"""


def test_every_width_has_a_kernel_and_every_kernel_a_width(tmp_path):
    """The host rule that maps rows onto threads, for all widths that stay on the chip and some beyond: rows are covered, fit the
    limits, and go to the slots and clusters that kernels are compiled for, all of which occur."""
    src, exe = tmp_path / "shapes.cu", tmp_path / "shapes"
    src.write_text(SHAPES_PROGRAM)
    r = subprocess.run([trbuild._nvcc(), *trbuild.ARCH, "-O1", "-std=c++17", "--expt-relaxed-constexpr", f"-I{trbuild.INCLUDE}",
                        f"-I{trbuild.CSRC}", str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([os.fspath(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


# ---- lists ---------------------------------------------------------------------

def call_list(f, ptrs, outs=None, numels=None, codes=None, count=None, norm=at(40), ws=at(50), ws_bytes=1 << 16, kind=0,
              max_norm=1.0, eps=1e-6):
    numels = [16] * len(ptrs) if numels is None else numels
    codes = [0] * len(ptrs) if codes is None else codes
    p, n, d = array.array("Q", ptrs), array.array("q", numels), array.array("i", codes)
    o = None if outs is None else array.array("Q", outs)
    a = lambda v: None if v is None else v.buffer_info()[0]  # noqa: E731
    count = len(ptrs) if count is None else count
    L = tr.load()
    if f == "norm":
        return L.tr_global_norm(kind, a(p), a(n), a(d), count, norm, ws, ws_bytes, None)
    if f == "by":
        return L.tr_clip_by_norm(a(p), a(o), a(n), a(d), count, norm, max_norm, eps, None)
    return L.tr_clip_global_norm(kind, a(p), a(o), a(n), a(d), count, max_norm, eps, norm, ws, ws_bytes, None)


@pytest.mark.parametrize("f", ["norm", "by", "clip"])
@pytest.mark.parametrize("args", [
    dict(ptrs=[at(0)], norm=None), dict(ptrs=[at(0)], norm=at(40) + 2), dict(ptrs=[at(0)], count=-1),
    dict(ptrs=[0]), dict(ptrs=[at(0) + 2]), dict(ptrs=[at(0) + 1], codes=[1]), dict(ptrs=[at(0)], codes=[3]),
    dict(ptrs=[at(0)], numels=[-1]), dict(ptrs=[at(0)], numels=[(1 << 42) + 1]), dict(ptrs=[at(40) - 32]),
])
def test_lists_refuse(f, args):
    assert call_list(f, **args) == E
    assert tr.tr_last_error_message()


@pytest.mark.parametrize("f", ["norm", "clip"])
@pytest.mark.parametrize("args", [
    dict(ptrs=[at(0)], kind=2), dict(ptrs=[at(0)], ws=None), dict(ptrs=[at(0)], ws_bytes=64), dict(ptrs=[at(0)], ws=at(50) + 8),
    dict(ptrs=[at(50) + 4096]), dict(ptrs=[at(0)], norm=at(50)),
])
def test_norms_refuse(f, args):
    assert call_list(f, **args) == E


@pytest.mark.parametrize("f", ["by", "clip"])
@pytest.mark.parametrize("args", [
    dict(ptrs=[at(0)], max_norm=-1.0), dict(ptrs=[at(0)], max_norm=float("nan")), dict(ptrs=[at(0)], eps=-1.0),
    dict(ptrs=[at(0)], eps=float("inf")),
    dict(ptrs=[at(0), at(0)]),                                  # the same tensor twice, in place
    dict(ptrs=[at(0), at(0) + 60]),                             # one element shared
    dict(ptrs=[at(0), at(1)], outs=[at(2), at(2)]),             # two outputs in one place
    dict(ptrs=[at(0), at(1)], outs=[at(1), at(2)]),             # an output over another tensor
    dict(ptrs=[at(0)], outs=[at(0) + 4]), dict(ptrs=[at(0)], outs=[0]), dict(ptrs=[at(0)], outs=[at(1) + 2]),
    dict(ptrs=[at(0)], outs=[at(40) - 4]),
    dict(ptrs=[at(9), at(0), at(0) + 32], outs=[at(10), at(0), at(3)], numels=[4, 400, 8]),  # an input inside a written range
])
def test_clipping_refuses(f, args):
    assert call_list(f, **args) == E


def test_list_workspace():
    n = ctypes.c_size_t(0)
    f = tr.load().tr_global_norm_workspace_bytes
    assert f(0, ctypes.byref(n)) == OK and n.value > 0
    one = n.value
    assert f(1000, ctypes.byref(n)) == OK and n.value == one
    assert f(1001, ctypes.byref(n)) == OK and n.value > one
    assert f(-1, ctypes.byref(n)) == E and f((1 << 31) + 1, ctypes.byref(n)) == E and f(1, None) == E
    # clipping nothing by a norm that is there touches nothing
    assert call_list("by", []) == OK
    assert call_list("by", [0, 0], numels=[0, 0]) == OK


def test_helpers_refuse_host_tensors():
    import torch
    x = torch.zeros(2, 8)
    with pytest.raises(TypeError):
        tr.gated_residual_norm(x, x)
    with pytest.raises(TypeError):
        tr.gated_residual_norm_backward(x, x, x)
    one = torch.zeros(())
    for f in (tr.global_norm, lambda t: tr.clip_global_norm(t, 1.0), lambda t: tr.clip_by_norm(t, one, 1.0),
              lambda t: tr.global_norm([], out=one), lambda t: tr.clip_global_norm([], 1.0, norm_out=one),
              lambda t: tr.clip_by_norm([], one, 1.0)):
        with pytest.raises(TypeError):
            f([x])


def test_dense_means_one_range():
    import torch
    t = torch.zeros(4, 6, 8)
    dense = tr._dense
    assert dense(t) and dense(t.permute(2, 0, 1)) and dense(t[1:3]) and dense(torch.zeros(())) and dense(t[:, :0])
    assert not dense(t[:, ::2]) and not dense(t[:, :3]) and not dense(torch.zeros(1, 8).expand(4, 8))
    assert dense(t[:1].permute(2, 1, 0))


# ---- the float64 definitions against differences ---------------------------------

@pytest.mark.parametrize("kind", ["rmsnorm", "layernorm"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("groups", [0, 1, 3, 6])
def test_definition_gradients_by_differences(kind, post, pre, groups):
    """Central differences of step 1e-5 in float64: third derivatives of order one leave
    1e-10, cancellation 1e-16 / 1e-5 of a sum of order 10; 1e-7 of the sum's size covers both."""
    rng = np.random.default_rng(groups + 10 * post + 20 * pre)
    rows, cols, layer, step = 6, 9, kind == "layernorm", 1e-5
    v = lambda want, *shape: rng.normal(size=shape) if want else None  # noqa: E731
    p = dict(x=v(1, rows, cols), a=v(1, rows, cols), post_w=v(post, cols), post_b=v(post and layer, cols),
             gate=v(groups, groups, cols), pre_w=v(pre, cols), pre_b=v(pre and layer, cols))
    dy, dh = v(pre, rows, cols), v(1, rows, cols)
    tail = dict(eps=1e-5, kind=kind, post=post, pre=pre, rs=0.7, bs=1.3)

    def loss(**k):
        (y, _), (h, _) = block.forward(**{**p, **k}, **tail)
        return (h * dh).sum() + ((y * dy).sum() if pre else 0.0)

    h = block.forward(**p, **tail)[1][0]
    g = block.backward(h, p["a"], dy, dh, p["post_w"], p["post_b"], p["gate"], p["pre_w"], **tail)
    names = dict(x="dx", a="dbranch", post_w="dpost_weight", post_b="dpost_bias", gate="dgate", pre_w="dweight", pre_b="dbias")
    assert set(g) == {names[k] for k, t in p.items() if t is not None}
    for k, t in p.items():
        if t is not None:
            d = rng.normal(size=t.shape)
            slope = (loss(**{k: t + step * d}) - loss(**{k: t - step * d})) / (2 * step)
            got = (g[names[k]][0] * d).sum()
            assert abs(slope - got) <= 1e-7 * (10 + np.abs(g[names[k]][0] * d).sum()), k
