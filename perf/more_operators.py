"""Cases that measure the operators at the two ends of a decoder: the embedding's lookup and its gradient, the layer norm
that stands behind it and in front of the head, and the head's softmax cross entropy, whose logits are never stored.

Each case is run either in its plain form (elementary torch operations in FP32, rounded once at the end) or, where
`own` is true, through the library's entry points. `exact` gives the same outputs from the definitions in FP64.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
E4M3_MAX = 448.0


def listed():
    """Widths and vocabularies are those of the library's own problems (4096, 8192, 131072, 50001) and odd ones between
    them."""
    return [
        # one decoding step's norm: a single row, where only latency counts
        {"name": "layer_norm_decode", "op": "norm", "rows": 1, "cols": 8192, "out": "bf16", "residual": True,
         "train": False},
        # a prompt's norm in front of an 8-bit product: the residual stream is updated, the operand leaves in 8 bits
        {"name": "layer_norm_e4m3_prompt", "op": "norm", "rows": 4000, "cols": 8192, "out": "e4m3", "residual": True,
         "train": False},
        # a training step of the norm, forward and backward
        {"name": "layer_norm_train", "op": "norm", "rows": 8192, "cols": 4096, "out": "bf16", "residual": True,
         "train": True},
        # the same at a width that no vector length divides, without a residual
        {"name": "layer_norm_train_odd", "op": "norm", "rows": 2001, "cols": 5123, "out": "bf16", "residual": False,
         "train": True},
        # the lookup of a decoding batch
        {"name": "embedding_decode", "op": "embedding", "tokens": 64, "vocab": 131072, "cols": 8192, "type": "bf16",
         "train": False, "base": False},
        # the lookup of packed prompts
        {"name": "embedding_prompt", "op": "embedding", "tokens": 16384, "vocab": 131072, "cols": 4096, "type": "bf16",
         "train": False, "base": False},
        # a training step's dense gradient of the table: most rows are zeros, a few tokens are very frequent
        {"name": "embedding_train", "op": "embedding", "tokens": 16384, "vocab": 131072, "cols": 4096, "type": "bf16",
         "train": True, "base": False},
        # tied weights: the head's gradient is there already and the lookup's is added; FP32, odd sizes
        {"name": "embedding_tied_odd", "op": "embedding", "tokens": 5003, "vocab": 50001, "cols": 1027, "type": "f32",
         "train": True, "base": True},
        # the loss of a single position: the head's bytes are the whole cost
        {"name": "loss_one_row", "op": "loss", "rows": 1, "vocab": 131072, "cols": 4096, "train": False},
        # scoring given text, an odd vocabulary, some places without a target
        {"name": "loss_scoring_odd", "op": "loss", "rows": 1500, "vocab": 50001, "cols": 2056, "train": False},
        # a training step of a small model, forward and backward, odd sizes
        {"name": "loss_train_small", "op": "loss", "rows": 300, "vocab": 8005, "cols": 520, "train": True},
        # a training step, forward and backward
        {"name": "loss_train", "op": "loss", "rows": 4096, "vocab": 131072, "cols": 4096, "train": True},
    ]


def _log_int(rng, lo, hi, multiple=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, -(-v // multiple) * multiple))


def draw(rng):
    op = rng.choice(("norm", "embedding", "loss"))
    if op == "norm":
        train = rng.random() < 0.5
        cols = _log_int(rng, 64, 16384, rng.choice((1, 8, 64)))
        return {"op": op, "rows": _log_int(rng, 1, min(16384, (1 << 26) // cols)), "cols": cols,
                "out": "bf16" if train else rng.choice(("bf16", "e4m3")), "residual": rng.random() < 0.6,
                "train": train}
    if op == "embedding":
        cols = _log_int(rng, 64, 8192, rng.choice((1, 8, 64)))
        return {"op": op, "tokens": _log_int(rng, 1, min(65536, (1 << 26) // cols)),
                "vocab": _log_int(rng, 1000, min(262144, (1 << 29) // cols)), "cols": cols,
                "type": rng.choice(("bf16", "bf16", "f32")), "train": rng.random() < 0.6, "base": rng.random() < 0.5}
    cols, vocab = _log_int(rng, 128, 8192, 8), _log_int(rng, 1000, 262144)
    most = min(8192, (1 << 29) // vocab, (4096 * 131072 * 4096) // (cols * vocab))
    return {"op": op, "rows": _log_int(rng, 1, most), "vocab": vocab, "cols": cols, "train": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _ids(g, n, vocab):
    """Token ids as text has them: the k-th most frequent about 1/k of the time, the ranks spread over the vocabulary."""
    u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab)) - 1).long().clamp(0, vocab - 1)
    step = 7919
    while math.gcd(step, vocab) != 1:
        step += 2
    return (rank * step + 13) % vocab


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "norm":
        rows, cols = case["rows"], case["cols"]
        # a residual stream: rows of different magnitude with a mean of their own, a few large columns
        s["x"] = _normal(g, rows, cols)
        s["residual"] = None
        if case["residual"]:
            r = torch.randn(rows, cols, generator=g, device=DEV) * (0.5 + 4 * torch.rand(rows, 1, generator=g, device=DEV))
            r += torch.randn(rows, 1, generator=g, device=DEV)
            r[:, :: max(1, cols // 7)] *= 8
            s["residual"] = r.to(torch.bfloat16)
        s["weight"] = (1 + 0.2 * torch.randn(cols, generator=g, device=DEV)).to(torch.bfloat16)
        s["bias"] = _normal(g, cols, std=0.3)
        if case["train"]:
            s["dy"] = _normal(g, rows, cols)
            s["dsum"] = _normal(g, rows, cols, std=0.5) if case["residual"] else None
    elif case["op"] == "embedding":
        dtype = torch.bfloat16 if case["type"] == "bf16" else torch.float32
        n, vocab, cols = case["tokens"], case["vocab"], case["cols"]
        ids = _ids(g, n, vocab)
        # a padded place has no token
        s["tokens"] = torch.where(torch.rand(n, generator=g, device=DEV) < 0.05, -1, ids) if n > 8 else ids
        s["scale"] = math.sqrt(cols)
        if not case["train"]:
            s["table"] = _normal(g, vocab, cols, std=0.02, dtype=dtype)
        else:
            s["dy"] = _normal(g, n, cols, std=0.01, dtype=dtype)
            # the head's gradient, where the weights are tied
            s["base"] = _normal(g, vocab, cols, std=0.01, dtype=dtype) if case["base"] else None
    else:
        rows, vocab, cols = case["rows"], case["vocab"], case["cols"]
        ids = _ids(g, rows, vocab)
        s["head"] = _normal(g, vocab, cols, std=2 / math.sqrt(cols))
        # normed rows that lean towards their target's weights, some more than others
        lean = 4 * torch.rand(rows, 1, generator=g, device=DEV)
        s["x"] = (torch.randn(rows, cols, generator=g, device=DEV) + lean * s["head"][ids].float()).to(torch.bfloat16)
        # a padded place has no target
        s["targets"] = torch.where(torch.rand(rows, generator=g, device=DEV) < 0.05, -1, ids) if rows > 8 else ids
        if case["train"]:
            # the mean over the rows, weighted, and the gradient of a penalty on the normaliser
            s["dloss"] = (0.5 + torch.rand(rows, generator=g, device=DEV)) / rows
            s["dlse"] = torch.randn(rows, generator=g, device=DEV) * (0.02 / rows)
    return s


# ---------------------------------------------------------------- plain forms (FP32)


def _plain_norm(s, out, train):
    x = s["x"].float()
    total = x if s["residual"] is None else (x + s["residual"].float()).to(torch.bfloat16).float()
    mean = total.mean(1, keepdim=True)
    c = total - mean
    rstd = torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)
    xh, w = c * rstd, s["weight"].float()
    y = xh * w + s["bias"].float()
    got = {} if s["residual"] is None else {"sum": total.to(torch.bfloat16)}
    if out == "bf16":
        got["y"] = y.to(torch.bfloat16)
    else:
        scale = y.abs().amax(1) / E4M3_MAX
        got["scale"] = scale
        got["y"] = (y / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    if train:
        dy = s["dy"].float()
        d = dy * w
        dx = rstd * (d - d.mean(1, keepdim=True) - xh * (d * xh).mean(1, keepdim=True))
        if s["dsum"] is not None:
            dx = dx + s["dsum"].float()
        got["dx"], got["dw"], got["db"] = dx.to(torch.bfloat16), (dy * xh).sum(0), dy.sum(0)
    return got


def _plain_embedding(s, case):
    tokens = s["tokens"]
    given = tokens >= 0
    if not case["train"]:
        rows = s["table"][tokens.clamp(min=0)].float() * s["scale"]
        return {"y": torch.where(given[:, None], rows, 0.0).to(s["table"].dtype)}
    dy = torch.where(given[:, None], s["dy"].float() * s["scale"], 0.0)
    total = torch.zeros(case["vocab"], case["cols"], device=DEV) if s["base"] is None else s["base"].float()
    return {"dtable": total.index_add(0, tokens.clamp(min=0), dy).to(s["dy"].dtype)}


def _plain_loss(s, case):
    x, w, targets = s["x"].float(), s["head"].float(), s["targets"]
    z = x @ w.T
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    lse = m + torch.log(total)
    given, at = targets >= 0, targets.clamp(min=0)[:, None]
    got = {"loss": torch.where(given, (lse - z.gather(1, at))[:, 0], 0.0), "lse": lse[:, 0]}
    if case["train"]:
        del z
        dloss = torch.where(given, s["dloss"], 0.0)[:, None]
        d = e.div_(total).mul_(dloss + s["dlse"][:, None])
        d.scatter_add_(1, at, -dloss)
        got["dx"], got["dhead"] = (d @ w).to(torch.bfloat16), (d.T @ x).to(torch.bfloat16)
    return got


# ---------------------------------------------------------------- one pass


def run(s):
    case = s["case"]
    if not own:
        if case["op"] == "norm":
            return _plain_norm(s, case["out"], case["train"])
        return _plain_embedding(s, case) if case["op"] == "embedding" else _plain_loss(s, case)

    import dense_tensor_core_persistent_gb300 as g

    if case["op"] == "norm":
        n = g.layer_norm(s["x"], s["weight"], s["bias"], residual=s["residual"], eps=EPS, out=case["out"],
                         save=case["train"])
        got = {"y": n.y} if s["residual"] is None else {"y": n.y, "sum": n.sum}
        if case["out"] == "e4m3":
            got["scale"] = n.scales
        if case["train"]:
            got["dx"], got["dw"], got["db"] = g.layer_norm_backward(s["dy"], n.sum, s["weight"], n.mean, n.rstd,
                                                                    dsum=s["dsum"])
        return got
    if case["op"] == "embedding":
        if not case["train"]:
            return {"y": g.embedding(s["table"], s["tokens"], scale=s["scale"])}
        return {"dtable": g.embedding_backward(s["dy"], s["tokens"], case["vocab"], scale=s["scale"], base=s["base"])}
    r = g.cross_entropy(s["x"], s["head"], s["targets"])
    got = {"loss": r.loss, "lse": r.lse}
    if case["train"]:
        got["dx"], got["dhead"] = g.cross_entropy_backward(s["x"], s["head"], s["targets"], r.lse, s["dloss"],
                                                           dlse=s["dlse"])
    return got


def work(case):
    """Bytes and operations of one pass that the definitions ask for."""
    if case["op"] == "norm":
        n, r = case["rows"] * case["cols"], 1 if case["residual"] else 0
        size = n * (2 + 4 * r + (1 if case["out"] == "e4m3" else 2)) + 4 * case["cols"]
        size += 4 * case["rows"] if case["out"] == "e4m3" else 0
        if case["train"]:
            size += n * (2 + 2 + 2 + 2 * r) + 10 * case["cols"]
        return {"bytes": size, "flops": n * (22 if case["train"] else 9)}
    if case["op"] == "embedding":
        b = 2 if case["type"] == "bf16" else 4
        n, v = case["tokens"] * case["cols"], case["vocab"] * case["cols"]
        size = 8 * case["tokens"] + (n * b + (2 * v * b if case["base"] else v * b) if case["train"] else 2 * n * b)
        return {"bytes": size, "flops": n * (2 if case["train"] else 1)}
    m, v, k = case["rows"], case["vocab"], case["cols"]
    size = 2 * (m * k + v * k) + 16 * m
    if case["train"]:
        size += 2 * (m * k + v * k) + 8 * m
    return {"bytes": size, "flops": (6 if case["train"] else 2) * m * v * k + 4 * m * v}


# ---------------------------------------------------------------- the definitions in FP64


def _round_e4m3(v):
    """FP64 values to the nearest E4M3 number (ties to even)."""
    a = v.abs().clamp(max=448.0)
    step = torch.exp2((torch.frexp(a).exponent.double() - 1).clamp(min=-6) - 3)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), v)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        t = s["x"].double()
        if s["residual"] is not None:
            t = (t + s["residual"].double()).to(torch.bfloat16).double()
        var, mean = torch.var_mean(t, 1, correction=0, keepdim=True)
        std = (var + EPS).sqrt()
        xh = (t - mean) / std
        y = torch.addcmul(s["bias"].double(), xh, s["weight"].double())
        got = {"y": y} if s["residual"] is None else {"y": y, "sum": t}
        if case["out"] == "e4m3":
            got["scale"] = y.abs().amax(1) / 448
            got["y"] = _round_e4m3(y / got["scale"][:, None])
        if case["train"]:
            dy = s["dy"].double()
            d = dy * s["weight"].double()
            n = case["cols"]
            got["dx"] = (n * d - d.sum(1, keepdim=True) - xh * (d * xh).sum(1, keepdim=True)) / (n * std)
            if s["dsum"] is not None:
                got["dx"] += s["dsum"].double()
            got["dw"], got["db"] = torch.einsum("rc,rc->c", dy, xh), torch.einsum("rc->c", dy)
        return got
    if case["op"] == "embedding":
        keep = (s["tokens"] >= 0).nonzero()[:, 0]
        ids = s["tokens"][keep]
        if not case["train"]:
            y = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device=DEV)
            y[keep] = s["table"].index_select(0, ids).double() * s["scale"]
            return {"y": y}
        total = (torch.zeros(case["vocab"], case["cols"], dtype=torch.float64, device=DEV) if s["base"] is None
                 else s["base"].double())
        return {"dtable": total.index_put_((ids,), s["dy"][keep].double() * s["scale"], accumulate=True)}
    m, v, k = case["rows"], case["vocab"], case["cols"]
    if (6 if case["train"] else 2) * m * v * k > 14e12:
        return None
    x, w = s["x"].double(), s["head"].double()
    logp = torch.mm(x, w.T)
    lse = torch.logsumexp(logp, 1)
    logp.sub_(lse[:, None])
    rows = (s["targets"] >= 0).nonzero()[:, 0]
    ids = s["targets"][rows]
    loss = torch.zeros(m, dtype=torch.float64, device=DEV)
    loss[rows] = -logp[rows, ids]
    got = {"loss": loss, "lse": lse}
    if case["train"]:
        dloss = torch.zeros(m, dtype=torch.float64, device=DEV)
        dloss[rows] = s["dloss"][rows].double()
        d = logp.exp_().mul_((dloss + s["dlse"].double())[:, None])
        d[rows, ids] -= dloss[rows]
        got["dx"], got["dhead"] = torch.mm(d, w), torch.mm(d.T, x)
    return got
