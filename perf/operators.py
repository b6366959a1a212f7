"""What is measured of the library's block norms and of its gradient clipping.

Four operators of a training step and of a decoding step:

* ``fwd``   the end of one block and the start of the next:
            h = residual_scale x + branch_scale gate post(branch), y = pre(h);
* ``bwd``   its gradients: dx, dbranch and those of both norms and of the gate;
* ``norm``  the norm over a list of gradient tensors;
* ``clip``  the same norm, and every tensor scaled by min(1, max_norm / (norm + 1e-6)).

Activations and gradients come in float32, bfloat16 or float16; norm weights,
biases and gates are float32, as everywhere in the library.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5        # of the norms
CLIP_EPS = 1e-6   # of the clipping factor
LARGEST = 16384 * 4096  # elements of the largest listed block case
LARGEST_LIST = 300_000_000  # elements of the longest drawn list of tensors
TYPES = ("f32", "bf16", "f16")


def _block(name, op, rows, cols, dtype, kind, gate_rows, post=True, pre=True, upstream=True, residual=1.0, branch=1.0):
    return {"name": name, "op": op, "rows": rows, "cols": cols, "dtype": dtype, "kind": kind, "gate_rows": gate_rows,
            "post": post, "pre": pre, "upstream": upstream, "residual_scale": residual, "branch_scale": branch}


def listed():
    return [
        # one new token of a decoder: latency is all that counts
        _block("fwd_1x4096_bf16", "fwd", 1, 4096, "bf16", "rmsnorm", 1),
        # a decoding batch without a gate, LayerNorm, in half precision
        _block("fwd_48x5120_f16", "fwd", 48, 5120, "f16", "layernorm", 0, branch=0.5),
        # the library's main benchmark shape
        _block("fwd_768x6144_f32", "fwd", 768, 6144, "f32", "rmsnorm", 1, residual=0.9, branch=0.25),
        # a training micro-batch of eight sequences of 2048 tokens, a gate for each sequence
        _block("fwd_16384x4096_bf16", "fwd", 16384, 4096, "bf16", "rmsnorm", 8),
        # the library's odd width: no row but the first starts on 16 bytes
        _block("bwd_37x1537_f32", "bwd", 37, 1537, "f32", "layernorm", 1),
        # the main shape: a branch with a gate for each channel and no norm of its own
        _block("bwd_768x6144_f32", "bwd", 768, 6144, "f32", "rmsnorm", 1, post=False, residual=0.9, branch=0.25),
        # three sequences of odd length in one batch, LayerNorm with all its column gradients
        _block("bwd_6039x2560_f16", "bwd", 6039, 2560, "f16", "layernorm", 3, branch=0.5),
        # the training micro-batch's backward
        _block("bwd_16384x4096_bf16", "bwd", 16384, 4096, "bf16", "rmsnorm", 8),
        # the gradients of adapters beside a frozen model: many small tensors
        {"name": "norm_small_f32", "op": "norm", "norm": "l2", "dtype": "f32", "layers": 0, "hidden": 0, "vocab": 0,
         "count": 48, "smallest": 1024, "largest": 65536, "sizes": 1},
        # a model whose matrices have bfloat16 gradients and whose vectors have float32 ones
        {"name": "norm_model_mixed", "op": "norm", "norm": "l2", "dtype": "mixed", "layers": 12, "hidden": 2048,
         "vocab": 50257, "count": 0, "smallest": 0, "largest": 0, "sizes": 0},
        # a small model in float32: its gradients fit the second-level cache
        {"name": "clip_small_f32", "op": "clip", "norm": "l2", "dtype": "f32", "layers": 6, "hidden": 512,
         "vocab": 5003, "count": 0, "smallest": 0, "largest": 0, "sizes": 0, "packed": False, "max_norm": 1.0},
        # a model's bfloat16 gradients clipped into the optimizer's flat buffer
        {"name": "clip_model_bf16", "op": "clip", "norm": "l2", "dtype": "bf16", "layers": 12, "hidden": 2048,
         "vocab": 50257, "count": 0, "smallest": 0, "largest": 0, "sizes": 0, "packed": False, "max_norm": 1.0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("fwd", "fwd", "bwd", "bwd", "norm", "clip"))
    dtype = rng.choice(TYPES)
    if op in ("fwd", "bwd"):
        cols = _log(rng, 64, 16384)
        if rng.random() < 0.6:  # most widths are multiples of 64; the others are what they are
            cols = max(64, cols // 64 * 64)
        rows = _log(rng, 1, min(16384, LARGEST // 2 // cols))
        divisors = [d for d in range(1, rows + 1) if rows % d == 0]
        gate = rng.choice((0, 1, divisors[len(divisors) // 2], rng.choice(divisors)))
        post, pre = rng.choice(((True, True), (True, True), (False, True), (True, False)))
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "kind": rng.choice(("rmsnorm", "layernorm")),
                "gate_rows": gate, "post": post, "pre": pre, "upstream": not pre or rng.random() < 0.8,
                "residual_scale": rng.choice((1.0, 0.7)), "branch_scale": rng.choice((1.0, 0.5))}
    case = {"op": op, "norm": rng.choice(("l2", "l2", "max")), "dtype": rng.choice(TYPES + ("mixed",)) if op == "norm" else dtype,
            "layers": 0, "hidden": 0, "vocab": 0, "count": _log(rng, 1, 400), "smallest": rng.choice((1, 7, 64, 1000)),
            "sizes": rng.randrange(1 << 20)}
    case["largest"] = max(case["smallest"] + 1, min(_log(rng, 1000, 50_000_000), LARGEST_LIST // case["count"]))
    if op == "clip":
        case["packed"] = rng.random() < 0.4  # the tensors back to back in the buffer, or each on 16 bytes
        case["max_norm"] = rng.choice((1.0, 1.0, 0.1, 1e6))
    return case


def _shapes(case):
    """The shapes of a case's list of tensors, the embedding first where there is one."""
    if case["layers"]:
        d = case["hidden"]
        layer = [(3 * d, d), (3 * d,), (d, d), (d,), (4 * d, d), (4 * d,), (d, 4 * d), (d,), (d,), (d,)]
        return [(case["vocab"], d)] + layer * case["layers"] + [(d,)]
    r = random.Random(case["sizes"])
    return [(_log(r, case["smallest"], case["largest"]),) for _ in range(case["count"])]


def _generator(seed):
    g = torch.Generator(device="cuda" if torch.cuda.is_available() else "cpu")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, scale=1.0, mean=0.0):
    t = torch.empty(shape, device=g.device, dtype=dtype)
    return t.normal_(mean, scale, generator=g)


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case}
    if case["op"] in ("fwd", "bwd"):
        rows, cols, dtype = case["rows"], case["cols"], DTYPES[case["dtype"]]
        layer = case["kind"] == "layernorm"
        vector = lambda mean, scale: _normal(g, (cols,), torch.float32, scale, mean)  # noqa: E731
        s["branch"] = _normal(g, (rows, cols), dtype, 0.5, 0.1)
        s["post_weight"] = vector(1.0, 0.2) if case["post"] else None
        s["post_bias"] = vector(0.0, 0.3) if case["post"] and layer else None
        s["weight"] = vector(1.0, 0.2) if case["pre"] else None
        s["bias"] = vector(0.0, 0.3) if case["pre"] and layer else None
        s["gate"] = _normal(g, (case["gate_rows"], cols), torch.float32, 0.5, 0.5) if case["gate_rows"] else None
        s["out"] = torch.empty((rows, cols), device=g.device, dtype=dtype)
        s["out2"] = torch.empty((rows, cols), device=g.device, dtype=dtype)
        if case["op"] == "fwd":
            s["x"] = _normal(g, (rows, cols), dtype, 2.0)
        else:
            s["h"] = _normal(g, (rows, cols), dtype, 2.0, 0.2)
            s["dy"] = _normal(g, (rows, cols), dtype, 1.0) if case["pre"] else None
            s["dh"] = _normal(g, (rows, cols), dtype, 0.5) if case["upstream"] else None
        return s
    shapes = _shapes(case)
    tensors = []
    for i, shape in enumerate(shapes):
        name = case["dtype"] if case["dtype"] != "mixed" else ("bf16" if len(shape) == 2 or i % 2 else "f32")
        t = _normal(g, shape, DTYPES[name], 1e-2 * 2.0 ** (i % 5))
        if len(shape) == 2 and i == 0 and case["vocab"]:  # tokens that were not in the batch have no gradient
            t[torch.rand(shape[0], generator=g, device=g.device) < 0.7] = 0
        tensors.append(t)
    s["tensors"] = tensors
    if case["op"] == "clip":
        dtype = DTYPES[case["dtype"]]
        step = 1 if case["packed"] else 16 // BYTES[case["dtype"]]
        pieces, at, starts = [], 0, []
        for t in tensors:
            starts.append(at)
            pad = -t.numel() % step
            pieces += [t, torch.zeros(pad, device=g.device, dtype=dtype)]
            at += t.numel() + pad
        s["pieces"] = pieces  # the tensors with the gaps between them in the flat buffer
        s["flat"] = torch.zeros(at, device=g.device, dtype=dtype)
        s["views"] = [s["flat"][b:b + t.numel()].view(t.shape) for b, t in zip(starts, tensors)]
    return s


def _unit(v, layer):
    """(v normalised, 1 / its scale) of every row, in 32 bits."""
    c = v - v.mean(1, keepdim=True) if layer else v
    r = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
    return c * r, r


def _grouped(gate, rows):
    """The gate of every row (one for all: as it is)."""
    return gate if gate.shape[0] in (1, rows) else gate.repeat_interleave(rows // gate.shape[0], 0)


def _group_sum(v, groups):
    return v.view(groups, -1, v.shape[1]).sum(1)


def _plain_fwd(s):
    c = s["case"]
    layer = c["kind"] == "layernorm"
    x, n = s["x"].float(), s["branch"].float()
    if c["post"]:
        n = _unit(n, layer)[0] * s["post_weight"]
        if layer:
            n = n + s["post_bias"]
    if s["gate"] is not None:
        n = n * _grouped(s["gate"], c["rows"])
    h = c["residual_scale"] * x + c["branch_scale"] * n
    out = {"h": h.to(s["x"].dtype)}
    if c["pre"]:
        y = _unit(h, layer)[0] * s["weight"]
        out["y"] = (y + s["bias"] if layer else y).to(s["x"].dtype)
    return out


def _plain_norm_bwd(unit, r, g, layer):
    """The gradient of unit(v) against v, given that of unit."""
    d = g - unit * (g * unit).mean(1, keepdim=True)
    return r * (d - g.mean(1, keepdim=True) if layer else d)


def _plain_bwd(s):
    c = s["case"]
    layer, groups = c["kind"] == "layernorm", c["gate_rows"]
    out = {}
    total = s["dh"].float() if s["dh"] is not None else 0.0
    if c["pre"]:
        unit, r = _unit(s["h"].float(), layer)
        dy = s["dy"].float()
        out["dweight"] = (dy * unit).sum(0)
        if layer:
            out["dbias"] = dy.sum(0)
        total = total + _plain_norm_bwd(unit, r, dy * s["weight"], layer)
    out["dx"] = (c["residual_scale"] * total).to(s["h"].dtype)
    total = c["branch_scale"] * total
    a = s["branch"].float()
    unit, r = _unit(a, layer) if c["post"] else (a, None)
    if groups:
        n = unit * s["post_weight"] if c["post"] else unit
        if c["post"] and layer:
            n = n + s["post_bias"]
        out["dgate"] = _group_sum(total * n, groups)
        total = total * _grouped(s["gate"], c["rows"])
    if c["post"]:
        out["dpost_weight"] = (total * unit).sum(0)
        if layer:
            out["dpost_bias"] = total.sum(0)
        total = _plain_norm_bwd(unit, r, total * s["post_weight"], layer)
    out["dbranch"] = total.to(s["h"].dtype)
    return out


def _plain_total(flat, kind):
    return flat.abs().max() if kind == "max" else torch.sqrt((flat * flat).sum())


def _plain_clip(s):
    c = s["case"]
    flat = torch.cat([t.reshape(-1) for t in s["pieces"]]).float()
    norm = _plain_total(flat, c["norm"])
    factor = torch.clamp(c["max_norm"] / (norm + CLIP_EPS), max=1.0)
    return {"norm": norm, "flat": (flat * factor).to(s["flat"].dtype)}


def _own_fwd(tr, s):
    c = s["case"]
    y, h = tr.gated_residual_norm(s["x"], s["branch"], s["post_weight"], s["post_bias"], s["gate"], s["weight"], s["bias"],
                                  eps=EPS, kind=c["kind"], post=c["post"], pre=c["pre"],
                                  residual_scale=c["residual_scale"], branch_scale=c["branch_scale"],
                                  out=s["out"] if c["pre"] else None, h_out=s["out2"])
    return {"h": h, "y": y} if c["pre"] else {"h": h}


def _own_bwd(tr, s):
    c = s["case"]
    g = tr.gated_residual_norm_backward(s["h"], s["branch"], s["dy"], s["dh"], s["post_weight"], s["post_bias"], s["gate"],
                                        s["weight"], eps=EPS, kind=c["kind"], post=c["post"], pre=c["pre"],
                                        residual_scale=c["residual_scale"], branch_scale=c["branch_scale"],
                                        dx=s["out"], dbranch=s["out2"])
    return {k: v for k, v in g._asdict().items() if v is not None}


def run(state):
    c = state["case"]
    if own:
        import fp32_row_reduction_gb300 as tr
        if c["op"] == "fwd":
            return _own_fwd(tr, state)
        if c["op"] == "bwd":
            return _own_bwd(tr, state)
        if c["op"] == "norm":
            return {"norm": tr.global_norm(state["tensors"], kind=c["norm"])}
        norm = tr.clip_global_norm(state["tensors"], c["max_norm"], kind=c["norm"], eps=CLIP_EPS, out=state["views"])
        return {"norm": norm, "flat": state["flat"]}
    if c["op"] == "fwd":
        return _plain_fwd(state)
    if c["op"] == "bwd":
        return _plain_bwd(state)
    if c["op"] == "norm":
        flat = torch.cat([t.reshape(-1) for t in state["tensors"]]).float()
        return {"norm": _plain_total(flat, c["norm"])}
    return _plain_clip(state)


def work(case):
    if case["op"] in ("fwd", "bwd"):
        n, cols, layer = case["rows"] * case["cols"], case["cols"], case["kind"] == "layernorm"
        vectors = (case["post"] + case["pre"]) * (1 + layer)
        if case["op"] == "fwd":
            tensors = 3 + case["pre"]                         # x, branch and h; y
            floats = vectors * cols + case["gate_rows"] * cols
            return {"bytes": n * tensors * BYTES[case["dtype"]] + 4 * floats, "flops": n * (6 + 4 * case["post"] + 4 * case["pre"])}
        # h and dy (pre), branch (its norm's or its gate's gradient), dh; dx and dbranch
        reads = 2 * case["pre"] + bool(case["post"] or case["gate_rows"]) + case["upstream"]
        floats = 2 * vectors * cols + 2 * case["gate_rows"] * cols
        return {"bytes": n * (reads + 2) * BYTES[case["dtype"]] + 4 * floats, "flops": n * (6 + 9 * case["post"] + 9 * case["pre"])}
    size = 0
    count = 0
    for i, shape in enumerate(_shapes(case)):
        name = case["dtype"] if case["dtype"] != "mixed" else ("bf16" if len(shape) == 2 or i % 2 else "f32")
        size += math.prod(shape) * BYTES[name]
        count += math.prod(shape)
    if case["op"] == "norm":
        return {"bytes": size + 4, "flops": 2 * count}
    return {"bytes": 2 * size + 4, "flops": 3 * count}


def _exact_norm(v, weight, bias, layer):
    """A norm of every row, from its definition."""
    if layer:
        mean = v.sum(1, keepdim=True) / v.shape[1]
        var = ((v - mean) ** 2).sum(1, keepdim=True) / v.shape[1]
        return (v - mean) / (var + EPS) ** 0.5 * weight + bias
    return v / ((v ** 2).sum(1, keepdim=True) / v.shape[1] + EPS) ** 0.5 * weight


def _exact_branch(a, s64, c):
    """branch_scale gate post(a), from its definition."""
    layer = c["kind"] == "layernorm"
    n = _exact_norm(a, s64["post_weight"], s64["post_bias"], layer) if c["post"] else a
    if s64["gate"] is not None:
        groups = torch.arange(c["rows"], device=a.device) // (c["rows"] // c["gate_rows"])
        n = n * s64["gate"][groups]
    return c["branch_scale"] * n


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "clip"):
        doubles = [t.double().reshape(-1) for t in (s["tensors"] if case["op"] == "norm" else s["pieces"]) if t.numel()]
        if case["norm"] == "max":
            norm = torch.stack([t.abs().max() for t in doubles]).max()
        else:
            norm = torch.stack([t @ t for t in doubles]).sum() ** 0.5
        if case["op"] == "norm":
            return {"norm": norm}
        factor = min(1.0, case["max_norm"] / (float(norm) + CLIP_EPS))
        return {"norm": norm, "flat": torch.cat([t * factor for t in doubles])}
    layer = case["kind"] == "layernorm"
    s64 = {k: v.double() if isinstance(v, torch.Tensor) and k not in ("out", "out2") else v for k, v in s.items()}
    for k in ("weight", "bias", "post_weight", "post_bias"):
        if s64[k] is None:
            s64[k] = torch.full((), 1.0 if k.endswith("weight") else 0.0, dtype=torch.float64, device=s["branch"].device)
    if case["op"] == "fwd":
        h = case["residual_scale"] * s64["x"] + _exact_branch(s64["branch"], s64, case)
        return {"h": h, "y": _exact_norm(h, s64["weight"], s64["bias"], layer)} if case["pre"] else {"h": h}
    # the gradients by differentiating the definition: first the pre-norm at h, then the branch
    out = {}
    total = s64["dh"] if s64["dh"] is not None else torch.zeros_like(s64["h"])
    if case["pre"]:
        leaves = [s64[k].requires_grad_() for k in (("h", "weight", "bias") if layer else ("h", "weight"))]
        grads = torch.autograd.grad(_exact_norm(s64["h"], s64["weight"], s64["bias"], layer), leaves, s64["dy"])
        total = total + grads[0]
        out["dweight"] = grads[1]
        if layer:
            out["dbias"] = grads[2]
    out["dx"] = case["residual_scale"] * total
    names = ["branch"] + (["post_weight"] + (["post_bias"] if layer else []) if case["post"] else []) + (["gate"] if case["gate_rows"] else [])
    grads = torch.autograd.grad(_exact_branch(s64["branch"].requires_grad_(), s64, case) if len(names) == 1 else
                                _exact_branch(*_leaves(s64, names), case), [s64[k] for k in names], total)
    out.update({"d" + k: v for k, v in zip(names, grads)})
    return out


def _leaves(s64, names):
    for k in names:
        s64[k].requires_grad_()
    return s64["branch"], s64
