"""Cases that measure the operators around the library's products: the RMS norm that makes their operands, the
gated feed-forward block, and the log probabilities read from the head's logits.

Each case is run either in its plain form (elementary torch operations in FP32, rounded once at the end) or, where
`own` is true, through the library's entry points. `exact` gives the same outputs from the definitions in FP64.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
E4M3_MAX = 448.0
E2M1_MAX = 6.0


def listed():
    """The sizes are those of the library's own problems (4000 x 14336 x 4096, 1 to 64 rows x 28672 x 8192, 8192 and
    4096 on a side) and odd ones between them."""
    return [
        # one decoding step's norm: a single row, where only latency counts
        {"name": "norm_decode", "op": "norm", "rows": 1, "cols": 8192, "out": "bf16", "residual": True, "train": False},
        # a prompt's norm in front of an 8-bit product: the residual stream is updated, the operand leaves in 8 bits
        {"name": "norm_e4m3_prompt", "op": "norm", "rows": 4000, "cols": 8192, "out": "e4m3", "residual": True,
         "train": False},
        # a training step of the norm, forward and backward, at a width that no vector length divides
        {"name": "norm_train_odd", "op": "norm", "rows": 4001, "cols": 4099, "out": "bf16", "residual": True,
         "train": True},
        # the norm that makes an NVFP4 product's operand, and that product
        {"name": "norm_nvfp4_product", "op": "norm_nvfp4", "M": 4000, "N": 14336, "K": 4096},
        # one decoding step of the gated block: the weights' bytes are the whole cost
        {"name": "glu_decode", "op": "glu", "M": 1, "N": 28672, "K": 8192, "act": "silu", "type": "bf16",
         "train": False},
        # a batch of decoding sequences with 8-bit weights and activations
        {"name": "glu_e4m3_batch", "op": "glu", "M": 64, "N": 28672, "K": 8192, "act": "silu", "type": "e4m3",
         "train": False},
        # a prompt of ragged length
        {"name": "glu_prompt", "op": "glu", "M": 4000, "N": 14336, "K": 4096, "act": "silu", "type": "bf16",
         "train": False},
        # a training step of a small block with odd sizes
        {"name": "glu_train_small", "op": "glu", "M": 300, "N": 1368, "K": 520, "act": "gelu_tanh", "type": "bf16",
         "train": True},
        # a training step, forward and backward
        {"name": "glu_train", "op": "glu", "M": 4096, "N": 14336, "K": 4096, "act": "silu", "type": "bf16",
         "train": True},
        # sampling: the chosen tokens' log probabilities and the alternatives, some of the vocabulary masked off
        {"name": "logprobs_decode", "op": "logprobs", "rows": 4, "vocab": 131072, "type": "bf16", "top": 20,
         "masked": True, "train": False},
        # scoring given text: FP32 logits, odd vocabulary
        {"name": "logprobs_scoring", "op": "logprobs", "rows": 1500, "vocab": 50001, "type": "f32", "top": 5,
         "masked": False, "train": False},
        # a policy's loss: log probabilities and entropy with their gradient
        {"name": "logprobs_train", "op": "logprobs", "rows": 4096, "vocab": 131072, "type": "bf16", "top": 0,
         "masked": False, "train": True},
    ]


def _log_int(rng, lo, hi, multiple=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, -(-v // multiple) * multiple))


def draw(rng):
    op = rng.choice(("norm", "norm", "glu", "glu", "glu", "logprobs", "logprobs", "norm_nvfp4"))
    if op == "norm":
        train = rng.random() < 0.4
        cols = _log_int(rng, 64, 16384, rng.choice((1, 8, 64)))
        return {"op": op, "rows": _log_int(rng, 1, min(16384, (1 << 26) // cols)), "cols": cols,
                "out": "bf16" if train else rng.choice(("bf16", "e4m3")), "residual": rng.random() < 0.7,
                "train": train}
    if op == "norm_nvfp4":
        return {"op": op, "M": _log_int(rng, 1, 4096), "N": _log_int(rng, 256, 14336, 8),
                "K": 256 * rng.randint(1, 32)}
    if op == "glu":
        kind = rng.choice(("bf16", "e4m3", "train"))
        mult = 16 if kind == "e4m3" else 8
        n, k = _log_int(rng, 128, 28672, mult), _log_int(rng, 128, 8192, mult)
        m = _log_int(rng, 1, max(1, min(8192, (4096 * 14336 * 4096) // (n * k))))
        return {"op": op, "M": m, "N": n, "K": k, "act": rng.choice(("silu", "gelu_tanh", "relu")),
                "type": "e4m3" if kind == "e4m3" else "bf16", "train": kind == "train"}
    vocab = _log_int(rng, 1000, 262144)
    kind = rng.choice(("bf16", "f32"))
    return {"op": op, "rows": _log_int(rng, 1, max(1, min(8192, (1 << 28) // vocab))), "vocab": vocab, "type": kind,
            "top": rng.choice((0, 1, 5, 20)), "masked": rng.random() < 0.3, "train": rng.random() < 0.4}


# ---------------------------------------------------------------- inputs


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _to_e4m3_rows(w):
    """Rows of FP32 values -> E4M3 codes and a scale a row."""
    scale = w.abs().amax(1) / E4M3_MAX
    return (w / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _nvfp4_weights(g, n, k):
    """Packed E2M1 codes and E4M3 scale bytes of a random weight matrix, as a quantiser leaves them."""
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.rand(n, k // 16, generator=g, device=DEV) * 0.02 + 0.01
    return codes, scales.to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] in ("norm", "norm_nvfp4"):
        rows, cols = (case["rows"], case["cols"]) if case["op"] == "norm" else (case["M"], case["K"])
        # a residual stream: rows of different magnitude, a few large columns
        s["x"] = _normal(g, rows, cols)
        s["residual"] = None
        if case.get("residual", True):
            r = torch.randn(rows, cols, generator=g, device=DEV) * (0.5 + 4 * torch.rand(rows, 1, generator=g, device=DEV))
            r[:, :: max(1, cols // 7)] *= 8
            s["residual"] = r.to(torch.bfloat16)
        s["weight"] = (1 + 0.2 * torch.randn(cols, generator=g, device=DEV)).to(torch.bfloat16)
        if case.get("train"):
            s["dy"] = _normal(g, rows, cols)
            s["dsum"] = _normal(g, rows, cols, std=0.5)
        if case["op"] == "norm_nvfp4":
            s["w"], s["w_scales"] = _nvfp4_weights(g, case["N"], case["K"])
    elif case["op"] == "glu":
        M, N, K = case["M"], case["N"], case["K"]
        x = torch.randn(M, K, generator=g, device=DEV)
        wg = torch.randn(N, K, generator=g, device=DEV) / math.sqrt(K)
        wu = torch.randn(N, K, generator=g, device=DEV) / math.sqrt(K)
        if case["type"] == "e4m3":
            s["x"], s["x_scale"] = _to_e4m3_rows(x)
            s["wg"], s["wg_scale"] = _to_e4m3_rows(wg)
            s["wu"], s["wu_scale"] = _to_e4m3_rows(wu)
        else:
            s["x"], s["wg"], s["wu"] = (t.to(torch.bfloat16) for t in (x, wg, wu))
        if case["train"]:
            s["dh"] = _normal(g, M, N)
    else:
        rows, vocab = case["rows"], case["vocab"]
        dtype = torch.bfloat16 if case["type"] == "bf16" else torch.float32
        logits = torch.randn(rows, vocab, generator=g, device=DEV)
        # rows from nearly uniform to sharply peaked
        logits *= 0.5 + 3 * torch.rand(rows, 1, generator=g, device=DEV)
        tokens = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
        if case["masked"]:
            off = torch.rand(rows, vocab, generator=g, device=DEV) < 0.25
            off.scatter_(1, tokens[:, None], False)
            logits.masked_fill_(off, -math.inf)
        s["logits"] = logits.to(dtype)
        # a padded place has no token
        s["tokens"] = torch.where(torch.rand(rows, generator=g, device=DEV) < 0.05, -1, tokens) if rows > 8 else tokens
        s["scale"] = 1.25 if case["top"] else 1.0
        if case["train"]:
            s["dlogprob"] = torch.randn(rows, generator=g, device=DEV)
            s["dentropy"] = torch.randn(rows, generator=g, device=DEV) * 0.1
    return s


# ---------------------------------------------------------------- plain forms (FP32)


def _plain_norm(s, out, train):
    x = s["x"].float()
    total = x if s["residual"] is None else (x + s["residual"].float()).to(torch.bfloat16).float()
    rstd = torch.rsqrt((total * total).mean(1, keepdim=True) + EPS)
    w = s["weight"].float()
    y = total * rstd * w
    got = {} if s["residual"] is None else {"sum": total.to(torch.bfloat16)}
    if out == "bf16":
        got["y"] = y.to(torch.bfloat16)
    else:
        scale = y.abs().amax(1) / E4M3_MAX
        got["scale"] = scale
        got["y"] = (y / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    if train:
        xh, dyw = total * rstd, s["dy"].float() * w
        dx = rstd * (dyw - xh * (dyw * xh).mean(1, keepdim=True)) + s["dsum"].float()
        got["dx"], got["dw"] = dx.to(torch.bfloat16), (s["dy"].float() * xh).sum(0)
    return got


def _e2m1_plain(v):
    """The nearest E2M1 value (0, 0.5, 1, 1.5, 2, 3, 4, 6; ties to the even code)."""
    a = v.abs().clamp(max=E2M1_MAX)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, v)


def _nvfp4_values(codes, scales, dtype):
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device, dtype=dtype)
    v = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), 2).flatten(1)
    return (v.view(v.shape[0], -1, 16) * scales.view(torch.float8_e4m3fn).to(dtype)[:, :, None]).flatten(1)


def _plain_norm_nvfp4(s):
    total = (s["x"].float() + s["residual"].float()).to(torch.bfloat16).float()
    y = total * torch.rsqrt((total * total).mean(1, keepdim=True) + EPS) * s["weight"].float()
    blocks = y.view(y.shape[0], -1, 16)
    sf = (blocks.abs().amax(2, keepdim=True) / E2M1_MAX).clamp(max=E4M3_MAX).to(torch.float8_e4m3fn).float()
    q = torch.where(sf > 0, _e2m1_plain(blocks / torch.where(sf > 0, sf, 1.0)) * sf, 0.0).flatten(1)
    return {"sum": total.to(torch.bfloat16), "c": (q @ _nvfp4_values(s["w"], s["w_scales"], torch.float32).T).to(torch.bfloat16)}


def _act_plain(g, act):
    """(act(g), act'(g))."""
    if act == "silu":
        sg = 1 / (1 + torch.exp(-g))
        return g * sg, sg * (1 + g * (1 - sg))
    if act == "relu":
        return g.clamp(min=0), (g > 0).to(g.dtype)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _plain_glu(s, case):
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    if case["type"] == "e4m3":
        x, wg, wu = x * s["x_scale"][:, None], wg * s["wg_scale"][:, None], wu * s["wu_scale"][:, None]
    g, u = x @ wg.T, x @ wu.T
    a, da = _act_plain(g, case["act"])
    got = {"h": (a * u).to(torch.bfloat16)}
    if case["train"]:
        dh = s["dh"].float()
        dg, du = dh * u * da, dh * a
        got["dx"] = (dg @ wg + du @ wu).to(torch.bfloat16)
        got["dwg"], got["dwu"] = (dg.T @ x).to(torch.bfloat16), (du.T @ x).to(torch.bfloat16)
    return got


def _plain_top(logits, top):
    """Indices of the `top` largest logits of each row, the lowest index first among equal ones."""
    bits = (logits + 0.0).view(torch.int32)  # (-0 counts as 0)
    order = torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF).long()
    place = 0xFFFFFFFF - torch.arange(logits.shape[1], device=logits.device)
    keys = torch.topk((order << 32) | place, top, dim=1).values
    return 0xFFFFFFFF - (keys & 0xFFFFFFFF)


def _plain_logprobs(s, case):
    logits, tokens = s["logits"].float(), s["tokens"]
    z = logits * s["scale"]
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    lse = m + torch.log(total)
    entropy = torch.log(total) - torch.where(e > 0, e * (z - m), 0.0).sum(1, keepdim=True) / total
    given = tokens >= 0
    at = tokens.clamp(min=0)[:, None]
    got = {"logprob": torch.where(given, (z.gather(1, at) - lse)[:, 0], 0.0), "entropy": entropy[:, 0], "lse": lse[:, 0]}
    if case["top"]:
        ids = _plain_top(logits, case["top"])
        got["top_logprobs"], got["top_ids"] = z.gather(1, ids) - lse, ids.to(torch.int32)
    if case["train"]:
        p, dlp, dh = e / total, torch.where(given, s["dlogprob"], 0.0)[:, None], s["dentropy"][:, None]
        dz = -dlp * p - dh * torch.where(p > 0, p * (z - lse + entropy), 0.0)
        dz.scatter_add_(1, at, dlp)
        got["dlogits"] = (dz * s["scale"]).to(s["logits"].dtype)
    return got


# ---------------------------------------------------------------- one pass


def run(s):
    case = s["case"]
    if not own:
        if case["op"] == "norm":
            return _plain_norm(s, case["out"], case["train"])
        if case["op"] == "norm_nvfp4":
            return _plain_norm_nvfp4(s)
        return _plain_glu(s, case) if case["op"] == "glu" else _plain_logprobs(s, case)

    import dense_tensor_core_persistent_gb300 as g

    if case["op"] == "norm":
        n = g.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, out=case["out"], save=case["train"])
        got = {"y": n.y} if s["residual"] is None else {"y": n.y, "sum": n.sum}
        if case["out"] == "e4m3":
            got["scale"] = n.scales
        if case["train"]:
            got["dx"], got["dw"] = g.rms_norm_backward(s["dy"], n.sum, s["weight"], n.rstd, dsum=s["dsum"])
        return got
    if case["op"] == "norm_nvfp4":
        n = g.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, out="nvfp4")
        return {"sum": n.sum, "c": g.matmul_nvfp4(n.y, n.scales, s["w"], s["w_scales"])}
    if case["op"] == "glu":
        if case["type"] == "e4m3":
            return {"h": g.glu_e4m3(s["x"], s["x_scale"], s["wg"], s["wg_scale"], s["wu"], s["wu_scale"], act=case["act"])}
        if not case["train"]:
            return {"h": g.glu_bf16(s["x"], s["wg"], s["wu"], act=case["act"])}
        h, saved = g.glu_bf16(s["x"], s["wg"], s["wu"], act=case["act"], save=True)
        dx, dwg, dwu = g.glu_bf16_backward(s["dh"], s["x"], s["wg"], s["wu"], saved, act=case["act"])
        return {"h": h, "dx": dx, "dwg": dwg, "dwu": dwu}
    r = g.token_logprobs(s["logits"], s["tokens"], top=case["top"], scale=s["scale"])
    got = {"logprob": r.logprob, "entropy": r.entropy, "lse": r.lse}
    if case["top"]:
        got["top_logprobs"], got["top_ids"] = r.top_logprobs, r.top_ids
    if case["train"]:
        got["dlogits"] = g.token_logprobs_backward(s["logits"], s["tokens"], r.lse, r.entropy, s["dlogprob"],
                                                   dentropy=s["dentropy"], scale=s["scale"])
    return got


def work(case):
    """Bytes and operations of one pass that the definitions ask for."""
    if case["op"] == "norm":
        n, r = case["rows"] * case["cols"], 1 if case["residual"] else 0
        size = n * (2 + 4 * r + (1 if case["out"] == "e4m3" else 2)) + 2 * case["cols"]
        size += 4 * case["rows"] if case["out"] == "e4m3" else 0
        if case["train"]:
            size += n * (2 + 2 + 2 + 2) + 6 * case["cols"]
        return {"bytes": size, "flops": n * (16 if case["train"] else 6)}
    if case["op"] == "norm_nvfp4":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 6 * M * K + 2 * K + N * K * 9 // 16 + 2 * M * N, "flops": 2 * M * N * K}
    if case["op"] == "glu":
        M, N, K = case["M"], case["N"], case["K"]
        b = 1 if case["type"] == "e4m3" else 2
        size = b * (M * K + 2 * N * K) + 2 * M * N + (4 * (M + 2 * N) if b == 1 else 0)
        if case["train"]:
            size += 2 * M * N + 2 * M * K + 4 * N * K
        return {"bytes": size, "flops": (12 if case["train"] else 4) * M * N * K}
    n, b = case["rows"] * case["vocab"], 2 if case["type"] == "bf16" else 4
    size = n * b * (2 if case["train"] else 1) + case["rows"] * (20 + 8 * case["top"])
    return {"bytes": size, "flops": n * (16 if case["train"] else 6)}


# ---------------------------------------------------------------- the definitions in FP64


def _round_binary(v, mantissa_bits, min_exp, largest):
    """FP64 values to the nearest number with `mantissa_bits` after the leading one (ties to even), subnormal below
    2**min_exp, limited to +-largest."""
    a = v.abs().clamp(max=largest)
    exp = torch.frexp(a).exponent.double() - 1
    step = torch.exp2(exp.clamp(min=min_exp) - mantissa_bits)
    return torch.copysign((torch.round(a / step) * step).clamp(max=largest), v)


def _exact_norm(s):
    total = s["x"].double()
    if s["residual"] is not None:
        total = (total + s["residual"].double()).to(torch.bfloat16).double()
    xh = total / (total.square().sum(1, keepdim=True) / total.shape[1] + EPS).sqrt()
    return total, xh, xh * s["weight"].double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        total, xh, y = _exact_norm(s)
        got = {"y": y} if s["residual"] is None else {"y": y, "sum": total}
        if case["out"] == "e4m3":
            got["scale"] = y.abs().amax(1) / 448
            got["y"] = _round_binary(y / got["scale"][:, None], 3, -6, 448.0)
        if case["train"]:
            rstd = xh.abs().sum(1, keepdim=True) / total.abs().sum(1, keepdim=True)
            d = s["dy"].double() * s["weight"].double()
            got["dx"] = rstd * d - rstd * xh * (d * xh).sum(1, keepdim=True) / total.shape[1] + s["dsum"].double()
            got["dw"] = torch.einsum("rc,rc->c", s["dy"].double(), xh)
        return got
    if case["op"] == "norm_nvfp4":
        total, _, y = _exact_norm(s)
        b = y.reshape(y.shape[0], -1, 16)
        sf = _round_binary(b.abs().amax(2, keepdim=True) / 6, 3, -6, 448.0)
        q = torch.where(sf > 0, _round_binary(b / sf.clamp(min=1e-300), 1, 0, 6.0) * sf, 0.0).reshape(y.shape)
        return {"sum": total, "c": q @ _nvfp4_values(s["w"], s["w_scales"], torch.float64).T}
    if case["op"] == "glu":
        x, wg, wu = s["x"].double(), s["wg"].double(), s["wu"].double()
        if case["type"] == "e4m3":
            x *= s["x_scale"].double()[:, None]
            wg *= s["wg_scale"].double()[:, None]
            wu *= s["wu_scale"].double()[:, None]
        g, u = torch.mm(x, wg.T), torch.mm(x, wu.T)
        if case["act"] == "silu":
            sg = torch.sigmoid(g)
            a, da = g * sg, sg + g * sg * (1 - sg)
        elif case["act"] == "relu":
            a, da = torch.relu(g), torch.heaviside(g, torch.zeros((), dtype=torch.float64, device=DEV))
        else:
            c = math.sqrt(2 / math.pi)
            t = torch.tanh(c * g * (1 + 0.044715 * g * g))
            a, da = g * (1 + t) / 2, (1 + t) / 2 + g * (1 - t * t) / 2 * c * (1 + 0.134145 * g * g)
        got = {"h": a * u}
        if case["train"]:
            dh = s["dh"].double()
            du = dh * a
            dg = dh * u * da
            got["dx"] = torch.mm(dg, wg).addmm_(du, wu)
            got["dwg"], got["dwu"] = torch.mm(dg.T, x), torch.mm(du.T, x)
        return got
    z = s["logits"].double() * s["scale"]
    lse = torch.logsumexp(z, 1, keepdim=True)
    logp = z - lse
    p = logp.exp()
    entropy = -(p * logp.clamp(min=-1e4)).sum(1, keepdim=True)
    given, at = s["tokens"] >= 0, s["tokens"].clamp(min=0)[:, None]
    got = {"logprob": logp.gather(1, at)[:, 0] * given, "entropy": entropy[:, 0], "lse": lse[:, 0]}
    if case["top"]:
        got["top_logprobs"], got["top_ids"] = torch.topk(logp, case["top"], dim=1).values, None
    if case["train"]:
        d = torch.zeros_like(p).scatter_(1, at, 1.0).sub_(p).mul_((s["dlogprob"].double() * given)[:, None])
        d -= s["dentropy"].double()[:, None] * p * (logp.clamp(min=-1e4) + entropy)
        got["dlogits"] = d * s["scale"]
    return got
