"""The block norms' definitions in float64, and rounding bounds for their binary32 kernels.

TEST INFRASTRUCTURE ONLY, like the rest of this package. Everything is numpy,
written from the formulas; the bounds follow each binary32 step of the formulas:

* u = 2^-24 is half a step of binary32, T half a step of the output's type;
* a sum whose longest chain has L additions is off by at most L u sum|terms|, L = 64
  for a row (at most 36 terms in binary32 in one thread, 10 tree levels, the terms' own
  roundings), and 128 + rows / 128 for a column;
* a mean square is then off by (L + 4) u of itself, 1 / sqrt(it + eps) by half of that and
  4 u more (division, root, their rounding), so by R = (L / 2 + 8) u of itself;
* products and sums add u of their value each.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
L = 64
R = (L / 2 + 8) * U
#: half a step of each type, and half its smallest step (below the normal range)
HALF_STEP = {"f32": (2.0 ** -24, 2.0 ** -150), "bf16": (2.0 ** -8, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25)}


def _one(v, like):
    return np.ones(like) if v is None else np.asarray(v, np.float64)


def _zero(v, like):
    return np.zeros(like) if v is None else np.asarray(v, np.float64)


def rows_gate(gate, rows, cols):
    """The gate of every row."""
    if gate is None:
        return np.ones((1, cols))
    gate = np.asarray(gate, np.float64).reshape(-1, cols)
    return np.repeat(gate, rows // gate.shape[0], 0) if rows else np.ones((0, cols))


def unit(v, kind, eps, err=0.0):
    """((v - mean) / sigma, 1 / sigma, the unit's bound) of every row, v being off by `err`."""
    layer = kind == "layernorm"
    mean = v.mean(1, keepdims=True) if layer else 0.0
    c = v - mean
    r = 1.0 / np.sqrt((c * c).mean(1, keepdims=True) + eps)
    hh = c * r
    shift = L * U * np.abs(v).mean(1, keepdims=True) + 2 * U * np.abs(v) if layer else 0.0
    e = err + (np.mean(err * np.ones_like(v), 1, keepdims=True) if layer else 0.0) + shift
    e = e * np.ones_like(v)
    return hh, r, r * (e + np.abs(hh) * (np.abs(hh) * e).mean(1, keepdims=True)) + np.abs(hh) * R


def rounded(v, err, dtype):
    """The bound of v once it is rounded to `dtype`."""
    step, tiny = HALF_STEP[dtype]
    return err + step * (np.abs(v) + err) + tiny


def forward(x, a, post_w, post_b, gate, pre_w, pre_b, eps, kind, post, pre, rs, bs):
    """((y, its bound), (h, its bound)), unrounded; y None without `pre`."""
    x, a = np.asarray(x, np.float64), np.asarray(a, np.float64)
    rows, cols = x.shape
    n, e = a, np.zeros_like(a)
    if post:
        w, b = _one(post_w, cols), _zero(post_b, cols)
        hh, _, eh = unit(a, kind, eps)
        n = hh * w + b
        e = np.abs(w) * eh + 2 * U * (np.abs(hh * w) + np.abs(b))
    g = rows_gate(gate, rows, cols)
    h = rs * x + bs * g * n
    e = np.abs(bs * g) * e + 4 * U * (np.abs(rs * x) + np.abs(bs * g * n))
    if not pre:
        return (None, None), (h, e)
    w, b = _one(pre_w, cols), _zero(pre_b, cols)
    hh, _, eh = unit(h, kind, eps, e)
    y = hh * w + b
    return (y, np.abs(w) * eh + 2 * U * (np.abs(hh * w) + np.abs(b))), (h, e)


def _norm_gradient(hh, e_hh, r, g, e_g, kind):
    """r (g - mean g - hh mean(g hh)) and its bound."""
    ag, ah = np.abs(g), np.abs(hh)
    m1, e1 = 0.0, 0.0
    if kind == "layernorm":
        m1 = g.mean(1, keepdims=True)
        e1 = e_g.mean(1, keepdims=True) + (L + 2) * U * ag.mean(1, keepdims=True)
    m2 = (g * hh).mean(1, keepdims=True)
    e2 = (e_g * ah + ag * e_hh).mean(1, keepdims=True) + (L + 4) * U * (ag * ah).mean(1, keepdims=True)
    t = g - m1 - hh * m2
    e = e_g + e1 + np.abs(m2) * e_hh + ah * e2 + 4 * U * (ag + np.abs(m1) + np.abs(hh * m2))
    return r * t, r * e + np.abs(r * t) * R + 2 * R * r * (ag + np.abs(m1) + np.abs(hh * m2))


def backward(h, a, dy, dh, post_w, post_b, gate, pre_w, eps, kind, post, pre, rs, bs):
    """{name: (gradient, bound)}, unrounded; names as in GatedResidualNormGrads."""
    a = np.asarray(a, np.float64)
    rows, cols = a.shape
    chain = (128 + rows / 128) * U
    out = {}
    d, e = _zero(dh, (rows, cols)), np.zeros((rows, cols))
    if pre:
        h, dy, w = np.asarray(h, np.float64), np.asarray(dy, np.float64), _one(pre_w, cols)
        hh, r, e_hh = unit(h, kind, eps)
        g = dy * w
        t, et = _norm_gradient(hh, e_hh, r, g, U * np.abs(g), kind)
        out["dweight"] = ((dy * hh).sum(0), (np.abs(dy) * e_hh).sum(0) + chain * np.abs(dy * hh).sum(0))
        if kind == "layernorm":
            out["dbias"] = (dy.sum(0), chain * np.abs(dy).sum(0))
        d, e = d + t, et + 2 * U * (np.abs(d) + np.abs(t))
    out["dx"] = (rs * d, abs(rs) * e + U * np.abs(rs * d))
    gates = rows_gate(gate, rows, cols)
    n, e_n, ah, e_ah, r = a, 0.0, a, 0.0, None
    w, b = _one(post_w if post else None, cols), _zero(post_b if post else None, cols)
    if post:
        ah, r, e_ah = unit(a, kind, eps)
        n, e_n = ah * w + b, np.abs(w) * e_ah
    if gate is not None:
        groups = np.asarray(gate).reshape(-1, cols).shape[0]
        fold = lambda v: v.reshape(groups, -1, cols).sum(1) if rows else np.zeros((groups, cols))  # noqa: E731
        size = np.abs(d) * (np.abs(ah * w) + np.abs(b))
        out["dgate"] = (bs * fold(d * n), abs(bs) * (fold(e * (np.abs(ah * w) + np.abs(b)) + np.abs(d) * e_n) + (chain + 4 * U) * fold(size)))
    q = bs * gates * d
    e_q = np.abs(bs * gates) * e + 2 * U * np.abs(q)
    if post:
        out["dpost_weight"] = ((q * ah).sum(0), (e_q * np.abs(ah) + np.abs(q) * e_ah).sum(0) + chain * np.abs(q * ah).sum(0))
        if kind == "layernorm":
            out["dpost_bias"] = (q.sum(0), e_q.sum(0) + chain * np.abs(q).sum(0))
        q, e_q = q * w, e_q * np.abs(w) + U * np.abs(q * w)
        out["dbranch"] = _norm_gradient(ah, e_ah, r, q, e_q, kind)
    else:
        out["dbranch"] = (q, e_q)
    return out
