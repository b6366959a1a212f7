"""What is measured of the vocabulary's two ends: the embedding at a model's start and the loss at its end.

Four operators of a training step, of scoring and of decoding:

* ``embed``       out[t] = scale table[ids[t]], zeros for an id outside the table;
* ``embed_grad``  its gradient, dtable[v] = scale (the sum of dy[t] over the tokens with ids[t] = v), dense;
* ``loss``        softmax cross entropy of logits = logit_scale hidden weight^T, which are
                  not kept: the loss of every row and its lse, the log of the sum of its exponentials;
* ``loss_grad``   from the saved lse and the gradients dloss of the losses (and dlse of the lse), the gradients
                  of hidden and weight, again without the logits.

Rows whose label is IGNORE have a loss and an lse of 0 and no gradient. Tables, weights and activations come in bfloat16 or
float16, those of the embedding in float32 too; losses, lse and their gradients are float32.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
IGNORE = -100
LARGEST = 8192 * 4096 * 50257     # products of the largest listed loss
LARGEST_TABLE = 50257 * 8192      # elements of the largest drawn table
LARGEST_TOKENS = 16384 * 4096     # elements of the largest drawn batch of embedded tokens
LOSS_SCALE = {"bf16": 1.0, "f16": 4096.0}  # half precision trains with scaled losses


def _embed(name, op, tokens, cols, vocab, dtype, grad="", spread="zipf", padded=0.0, scale=1.0):
    return {"name": name, "op": op, "tokens": tokens, "cols": cols, "vocab": vocab, "dtype": dtype, "grad": grad or dtype,
            "spread": spread, "padded": padded, "scale": scale}


def _loss(name, op, rows, cols, vocab, dtype, ignored=0.0, z=False, scale=1.0):
    return {"name": name, "op": op, "rows": rows, "cols": cols, "vocab": vocab, "dtype": dtype, "ignored": ignored, "z": z,
            "logit_scale": scale}


def listed():
    return [
        # one step of a decoding batch: a handful of rows of the table
        _embed("embed_48x5120_f16", "embed", 48, 5120, 50257, "f16", scale=71.5),
        # a padded batch of odd lengths at the library's odd width: no row but the first starts on 16 bytes
        _embed("embed_6039x1537_f32", "embed", 6039, 1537, 5003, "f32", padded=0.1),
        # a training micro-batch of eight sequences of 2048 tokens
        _embed("embed_16384x4096_bf16", "embed", 16384, 4096, 50257, "bf16", scale=64.0),
        # a small vocabulary trained on few tokens: most of the table has no gradient
        _embed("embed_grad_48x512_f32", "embed_grad", 48, 512, 5003, "f32"),
        # half-precision gradients of an odd width collected in float32, a padded batch
        _embed("embed_grad_6039x1537_f16", "embed_grad", 6039, 1537, 50257, "f16", grad="f32", padded=0.1),
        # the training micro-batch's backward; one token in sixteen is the most frequent one
        _embed("embed_grad_16384x4096_bf16", "embed_grad", 16384, 4096, 50257, "bf16", scale=64.0),
        # the loss of one new token: the table is read for a single row
        _loss("loss_1x4096_bf16", "loss", 1, 4096, 50257, "bf16"),
        # scoring a decoding batch
        _loss("loss_48x5120_f16", "loss", 48, 5120, 50257, "f16", scale=0.5),
        # a training micro-batch's forward
        _loss("loss_8192x4096_bf16", "loss", 8192, 4096, 50257, "bf16", ignored=0.1),
        # the library's odd width: rows that do not start on 16 bytes
        _loss("loss_grad_37x1537_f16", "loss_grad", 37, 1537, 5003, "f16"),
        # three sequences of odd length, half precision with a scaled loss, padding, and a gradient of the lse
        _loss("loss_grad_6039x2560_f16", "loss_grad", 6039, 2560, 50257, "f16", ignored=0.2, z=True),
        # the training micro-batch's backward
        _loss("loss_grad_8192x4096_bf16", "loss_grad", 8192, 4096, 50257, "bf16", ignored=0.1),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("embed", "embed_grad", "loss", "loss", "loss_grad", "loss_grad"))
    cols = _log(rng, 64, 8192)
    if rng.random() < 0.6:  # most widths are multiples of 64; the others are what they are
        cols = max(64, cols // 64 * 64)
    if op in ("embed", "embed_grad"):
        dtype = rng.choice(("f32", "bf16", "f16"))
        return {"op": op, "cols": cols, "vocab": _log(rng, 16, min(262144, LARGEST_TABLE // cols)),
                "tokens": _log(rng, 1, min(131072, LARGEST_TOKENS // cols)), "dtype": dtype,
                "grad": rng.choice((dtype, "f32")) if op == "embed_grad" else dtype, "spread": rng.choice(("zipf", "zipf", "even")),
                "padded": rng.choice((0.0, 0.0, 0.1, 0.5)), "scale": rng.choice((1.0, 1.0, math.sqrt(cols)))}
    vocab = _log(rng, 16, 131072)
    if rng.random() < 0.4:  # some vocabularies are padded to a multiple of 64
        vocab = max(64, vocab // 64 * 64)
    return {"op": op, "cols": cols, "vocab": vocab, "rows": _log(rng, 1, min(16384, LARGEST // cols // vocab)),
            "dtype": rng.choice(("bf16", "f16")), "ignored": rng.choice((0.0, 0.0, 0.1, 0.6)), "z": rng.random() < 0.4,
            "logit_scale": rng.choice((1.0, 1.0, 0.5, 2.0))}


def _generator(seed):
    g = torch.Generator(device="cuda" if torch.cuda.is_available() else "cpu")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, scale=1.0, mean=0.0):
    t = torch.empty(shape, device=g.device, dtype=dtype)
    return t.normal_(mean, scale, generator=g)


def _tokens(g, n, vocab, spread):
    """Token ids: evenly spread, or as in text, where the k-th token's share is as 1 / k."""
    u = torch.rand(n, generator=g, device=g.device, dtype=torch.float64)
    ids = vocab * u if spread == "even" else torch.exp(u * math.log(vocab + 1)) - 1
    return ids.long().clamp(0, vocab - 1)


def _masked(ids, share, value):
    """Some of the ids replaced by `value`, at the ends of four sequences."""
    if share:
        length = _length(ids.numel())
        at = torch.arange(ids.numel(), device=ids.device) % length
        ids[at >= length - int(share * length)] = value
    return ids


def _length(n):
    return max(1, -(-n // 4))


def _left(n, share):
    """How many of n ids _masked leaves."""
    length = _length(n)
    return sum(min(n - at, length - int(share * length)) for at in range(0, n, length))


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case}
    dtype = DTYPES[case["dtype"]]
    if case["op"] in ("embed", "embed_grad"):
        s["ids"] = _masked(_tokens(g, case["tokens"], case["vocab"], case["spread"]), case["padded"], -1)
        if case["op"] == "embed":
            s["table"] = _normal(g, (case["vocab"], case["cols"]), dtype, 0.02)
        else:
            s["dy"] = _normal(g, (case["tokens"], case["cols"]), dtype, 0.01)
            s["dtable"] = torch.empty((case["vocab"], case["cols"]), device=g.device, dtype=DTYPES[case["grad"]])
        return s
    rows, cols, vocab = case["rows"], case["cols"], case["vocab"]
    s["hidden"] = _normal(g, (rows, cols), dtype)  # what comes out of the last norm
    s["weight"] = _normal(g, (vocab, cols), dtype, 1.5 / math.sqrt(cols))
    s["labels"] = _masked(_tokens(g, rows, vocab, "zipf"), case["ignored"], IGNORE)
    if case["op"] == "loss_grad":
        s["lse"] = _plain_loss(s)["lse"]
        counted = max(1, int((s["labels"] != IGNORE).sum()))
        s["dloss"] = torch.full((rows,), LOSS_SCALE[case["dtype"]] / counted, device=g.device)  # of their mean
        s["dlse"] = 2e-3 * s["dloss"] * s["lse"] if case["z"] else None  # of 1e-3 lse^2, which keeps the logits small
        s["dhidden"] = torch.empty_like(s["hidden"])
        s["dweight"] = torch.empty_like(s["weight"])
    return s


def _plain_embed(s):
    ids, table = s["ids"], s["table"]
    inside = (ids >= 0) & (ids < table.shape[0])
    rows = table[ids.clamp(0, table.shape[0] - 1)].float() * s["case"]["scale"]
    return {"out": torch.where(inside[:, None], rows, 0.0).to(table.dtype)}


def _plain_embed_grad(s):
    ids, c = s["ids"], s["case"]
    inside = (ids >= 0) & (ids < c["vocab"])
    dy = torch.where(inside[:, None], s["dy"].float() * c["scale"], 0.0)
    sums = torch.zeros((c["vocab"], c["cols"]), device=dy.device)
    sums.index_add_(0, ids.clamp(0, c["vocab"] - 1), dy)
    return {"dtable": sums.to(s["dtable"].dtype)}


def _picked(labels, vocab):
    """(whether a row has a label, the label or 0)."""
    inside = (labels >= 0) & (labels < vocab)
    return inside, torch.where(inside, labels, 0)


def _plain_loss(s):
    c = s["case"]
    z = c["logit_scale"] * (s["hidden"].float() @ s["weight"].float().T)
    top = z.amax(1, keepdim=True)
    lse = torch.log(torch.exp(z - top).sum(1)) + top[:, 0]
    inside, label = _picked(s["labels"], c["vocab"])
    loss = lse - torch.where(inside, z.gather(1, label[:, None])[:, 0], 0.0)
    counted = s["labels"] != IGNORE
    return {"loss": torch.where(counted, loss, 0.0), "lse": torch.where(counted, lse, 0.0)}


def _plain_loss_grad(s):
    c = s["case"]
    hidden, weight = s["hidden"].float(), s["weight"].float()
    counted = s["labels"] != IGNORE
    dloss = torch.where(counted, s["dloss"], 0.0)
    total = dloss + torch.where(counted, s["dlse"], 0.0) if c["z"] else dloss
    dz = torch.where(counted[:, None], torch.exp(c["logit_scale"] * (hidden @ weight.T) - s["lse"][:, None]) * total[:, None], 0.0)
    inside, label = _picked(s["labels"], c["vocab"])
    dz[torch.arange(c["rows"], device=dz.device), label] -= torch.where(inside, dloss, 0.0)
    dz = dz * c["logit_scale"]
    return {"dhidden": (dz @ weight).to(s["hidden"].dtype), "dweight": (dz.T @ hidden).to(s["weight"].dtype)}


def run(state):
    c = state["case"]
    if own:
        import fp32_row_reduction_gb300 as tr
        if c["op"] == "embed":
            return {"out": tr.embedding(state["ids"], state["table"], scale=c["scale"])}
        if c["op"] == "embed_grad":
            return {"dtable": tr.embedding_backward(state["dy"], state["ids"], scale=c["scale"], dtable=state["dtable"])}
        if c["op"] == "loss":
            loss, lse = tr.linear_cross_entropy(state["hidden"], state["weight"], state["labels"],
                                                logit_scale=c["logit_scale"], ignore_label=IGNORE)
            return {"loss": loss, "lse": lse}
        dhidden, dweight = tr.linear_cross_entropy_backward(
            state["hidden"], state["weight"], state["labels"], state["lse"], state["dloss"], state["dlse"],
            logit_scale=c["logit_scale"], ignore_label=IGNORE, dhidden=state["dhidden"], dweight=state["dweight"])
        return {"dhidden": dhidden, "dweight": dweight}
    return {"embed": _plain_embed, "embed_grad": _plain_embed_grad, "loss": _plain_loss, "loss_grad": _plain_loss_grad}[c["op"]](state)


def work(case):
    if case["op"] in ("embed", "embed_grad"):
        tokens = _left(case["tokens"], case["padded"])
        n, table = case["tokens"] * case["cols"], case["vocab"] * case["cols"]
        if case["op"] == "embed":  # a row of the table is read once, however many tokens have it
            share = min(tokens, case["vocab"]) * case["cols"]
            return {"bytes": (share + n) * BYTES[case["dtype"]] + 8 * case["tokens"], "flops": tokens * case["cols"]}
        return {"bytes": tokens * case["cols"] * BYTES[case["dtype"]] + table * BYTES[case["grad"]] + 8 * case["tokens"],
                "flops": 2 * tokens * case["cols"]}
    # rows without a loss are neither read nor computed
    rows, cols, vocab, b = _left(case["rows"], case["ignored"]), case["cols"], case["vocab"], BYTES[case["dtype"]]
    if case["op"] == "loss":
        return {"bytes": (rows + vocab) * cols * b + 16 * case["rows"], "flops": 2 * rows * cols * vocab + 4 * rows * vocab}
    # the logits once more, and a product for each gradient
    return {"bytes": (rows + case["rows"] + 2 * vocab) * cols * b + (16 + 4 * case["z"]) * case["rows"],
            "flops": 6 * rows * cols * vocab + 5 * rows * vocab}


def _exact_loss(hidden, weight, labels, scale, vocab):
    z = scale * torch.mm(hidden, weight.t())
    lse = torch.logsumexp(z, 1)
    has = (labels >= 0) & (labels < vocab)
    chosen = torch.zeros_like(lse)
    chosen[has] = z[has, labels[has]]
    counted = (labels != IGNORE).double()
    return (lse - chosen) * counted, lse * counted


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "embed":
        out = torch.zeros((case["tokens"], case["cols"]), dtype=torch.float64, device=s["ids"].device)
        has = (s["ids"] >= 0) & (s["ids"] < case["vocab"])
        out[has] = s["table"].double()[s["ids"][has]] * case["scale"]
        return {"out": out}
    if case["op"] == "embed_grad":
        has = (s["ids"] >= 0) & (s["ids"] < case["vocab"])
        out = torch.zeros((case["vocab"], case["cols"]), dtype=torch.float64, device=s["ids"].device)
        out.index_put_((s["ids"][has],), s["dy"].double()[has], accumulate=True)
        return {"dtable": out * case["scale"]}
    # the gradients by differentiating the definition, a part of the rows at a time
    grad = case["op"] == "loss_grad"
    weight = s["weight"].double().requires_grad_(grad)
    parts = []
    dweight = torch.zeros_like(weight)
    for at in range(0, case["rows"], 4096):
        part = slice(at, min(at + 4096, case["rows"]))
        hidden, labels = s["hidden"][part].double().requires_grad_(grad), s["labels"][part]
        loss, lse = _exact_loss(hidden, weight, labels, case["logit_scale"], case["vocab"])
        if not grad:
            parts.append((loss, lse))
            continue
        total = (loss * s["dloss"][part]).sum()
        if case["z"]:
            total = total + (lse * s["dlse"][part]).sum()
        dh, dw = torch.autograd.grad(total, (hidden, weight))
        parts.append((dh,))
        dweight = dweight + dw
    if grad:
        return {"dhidden": torch.cat([p[0] for p in parts]), "dweight": dweight.detach()}
    return {"loss": torch.cat([p[0] for p in parts]), "lse": torch.cat([p[1] for p in parts])}
