"""The embedding and the linear cross entropy in float64, with rounding bounds for their kernels.

TEST INFRASTRUCTURE ONLY, like the rest of this package. Written from the formulas with torch in
float64 (on the tensors' own device); each function returns (value, bound of what a kernel may be off before
its last rounding). The bounds follow each step of the formulas:

* u = 2^-24 is half a step of binary32, T half a step of the 16-bit type (bf16 2^-8, f16 2^-11);
* products of two 16-bit numbers are exact in binary32 (8 + 8 or 11 + 11 bits), and a sum of n of them, in any order and
  grouping, rounds at most n partial sums, each no larger than sum |products|: n u sum |products| (also where sixteen products at a time are
  added and rounded toward zero, by 2 u at most). The kernels sum in parts and are far nearer; tests of long sums have bounds of their own;
* a row of logits is off by e = cols u sum |hidden weight|, its log-sum-exp by the largest e; 2^x is off by
  2^-21 of itself, the sums of exponentials by (64 + vocab / 64) u, the logarithm and the products with ln 2 and log2(e) by
  4 u of what they multiply;
* a probability is then off by e + 8 u (|logit| + |lse|) + 2^-20 of itself; dz is rounded to the type: T (its square where dz is taken in
  two terms), and half of the smallest step, 2^-25 for f16, after the largest coefficient, |dloss| + |dlse|, has been brought to 2^14 .. 2^15:
  2^-25 2^-14 of it at most, of which twice as much is allowed.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
HALF_STEP = {torch.float32: (2.0 ** -24, 2.0 ** -150), torch.bfloat16: (2.0 ** -8, 2.0 ** -134), torch.float16: (2.0 ** -11, 2.0 ** -25)}


def rounded(v, err, dtype):
    """The bound of v once it is rounded to `dtype`."""
    step, tiny = HALF_STEP[dtype]
    return err + step * (v.abs() + err) + tiny


def f32(v):
    """A Python number as the binary32 that a kernel is given."""
    return float(torch.tensor(v, dtype=torch.float32))


def embedding(ids, table, scale):
    t = table.double()
    inside = (ids >= 0) & (ids < table.shape[0])
    out = t[torch.where(inside, ids, 0)] * f32(scale)
    out = torch.where(inside[..., None], out, torch.zeros_like(out))
    return out, U * out.abs()


def embedding_backward(dy, ids, vocab, scale, base=None):
    """`base`: what the gradient is added to."""
    cols = dy.shape[-1]
    ids, dy = ids.reshape(-1), dy.reshape(-1, cols)
    inside = (ids >= 0) & (ids < vocab)
    ids, dy = ids[inside], dy[inside].double()
    sums = torch.zeros((vocab, cols), dtype=torch.float64, device=dy.device).index_add_(0, ids, dy)
    size = torch.zeros_like(sums).index_add_(0, ids, dy.abs())
    count = torch.zeros(vocab, dtype=torch.float64, device=dy.device).index_add_(0, ids, torch.ones_like(ids, dtype=torch.float64))
    # a chain: all of a short segment; of a long one, a tile of 32, an eighth of the tiles, and the eighths
    chain = torch.where(count <= 64, count, 48 + count / 256)[:, None]
    s = abs(f32(scale))
    out, err = f32(scale) * sums, s * (chain * U * size + U * sums.abs())
    if base is not None:
        out, err = out + base.double(), err + U * (out + base.double()).abs() + U * base.double().abs()
    return out, err


def logits(hidden, weight, scale):
    """(logits, their bound)."""
    h, w = hidden.double(), weight.double()
    z = f32(scale) * (h @ w.T)
    size = abs(f32(scale)) * (h.abs() @ w.abs().T)
    return z, (hidden.shape[1] + 4) * U * size


def linear_cross_entropy(hidden, weight, labels, scale=1.0, ignore=-100):
    """((losses, bound), (lse, bound)); rows without a loss may hold anything."""
    v = weight.shape[0]
    counted = labels != ignore
    z, e = logits(torch.where(counted[:, None], hidden, torch.zeros_like(hidden)), weight, scale)
    lse = torch.logsumexp(z, 1)
    inside = (labels >= 0) & (labels < v)
    label = torch.where(inside, labels, 0)[:, None]
    zero = torch.zeros_like(lse)
    picked = torch.where(inside, z.gather(1, label)[:, 0], zero)
    e_lse = e.amax(1) + 2.0 ** -20 + (64 + v / 64) * U + 8 * U * (z.abs().amax(1) + lse.abs())
    e_loss = e_lse + torch.where(inside, e.gather(1, label)[:, 0], zero) + 8 * U * picked.abs()
    keep = lambda t: torch.where(counted, t, zero)  # noqa: E731
    return (keep(lse - picked), keep(e_loss)), (keep(lse), keep(e_lse))


def linear_cross_entropy_backward(hidden, weight, labels, lse, dloss=None, dlse=None, scale=1.0, ignore=-100, terms=1):
    """((dhidden, bound), (dweight, bound)); `terms`: how many of the type dz is taken in, each rounding what those before it left."""
    dtype, v = hidden.dtype, weight.shape[0]
    counted = labels != ignore
    hidden = torch.where(counted[:, None], hidden, torch.zeros_like(hidden))
    z, e = logits(hidden, weight, scale)
    one = torch.ones(hidden.shape[0], dtype=torch.float64, device=hidden.device)
    d = torch.where(counted, one if dloss is None else dloss.double(), 0 * one)
    total = d + (torch.where(counted, dlse.double(), 0 * one) if dlse is not None else 0.0)
    lse = torch.where(counted, lse.double(), 0 * one)[:, None]
    p = total[:, None] * torch.exp(torch.where(counted[:, None], z - lse, torch.zeros_like(z)))
    p_err = p.abs() * (e + 8 * U * (z.abs() + lse.abs()) + 2.0 ** -20)
    inside = counted & (labels >= 0) & (labels < v)
    at = torch.nonzero(inside)[:, 0]
    dz = p.clone()
    dz[at, labels[at]] -= d[at]
    dz_err = p_err + 4 * U * p.abs()
    dz_err[at, labels[at]] += 2 * U * d[at].abs()
    step, tiny = HALF_STEP[dtype]
    most = float((d.abs() + (total - d).abs()).max()) if d.numel() else 0.0
    dz_err = dz_err + step ** terms * (dz.abs() + dz_err) + (tiny * 2 * most * 2.0 ** -14 if dtype == torch.float16 else 0.0)
    dz_err[~counted] = 0.0
    s = abs(f32(scale))
    h, w = hidden.double(), weight.double()
    size_h, size_w = dz.abs() @ w.abs(), dz.abs().T @ h.abs()
    dh, dw = f32(scale) * (dz @ w), f32(scale) * (dz.T @ h)
    dh_err = s * (dz_err @ w.abs() + (v + 8) * U * size_h)
    dw_err = s * (dz_err.T @ h.abs() + (h.shape[0] + 8) * U * size_w)
    return (dh, dh_err), (dw, dw_err)
