"""A decoder's feed-forward half and its head from the library's operators, as a serving step and as a training step.

    residual stream -> RMS norm -> gated block -> down product (+ residual) -> RMS norm -> head product -> log probabilities

`serve` picks the next tokens of a batch: the norm writes the residual stream and, in E4M3 with a scale per row, the
gated block's operand. `train_step` returns the mean log probability of given tokens plus an entropy bonus and the
gradient of every weight. Run it on a GPU:

    python examples/feed_forward.py --rows 64 --width 1024 --hidden 2816 --vocab 32000
"""
from __future__ import annotations

import argparse
import os
import sys
from typing import NamedTuple

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dense_tensor_core_persistent_gb300 as g  # noqa: E402

BF16 = torch.bfloat16


class Weights(NamedTuple):
    """norm, final_norm: width; gate, up: hidden x width; down: width x hidden; head: vocab x width (all BF16)."""
    norm: torch.Tensor
    gate: torch.Tensor
    up: torch.Tensor
    down: torch.Tensor
    final_norm: torch.Tensor
    head: torch.Tensor


def random_weights(width: int, hidden: int, vocab: int, device="cuda", seed: int = 0) -> Weights:
    gen = torch.Generator(device=device).manual_seed(seed)

    def matrix(rows, cols):
        return (torch.randn(rows, cols, generator=gen, device=device) / cols ** 0.5).to(BF16)

    return Weights(torch.ones(width, dtype=BF16, device=device), matrix(hidden, width), matrix(hidden, width),
                   matrix(width, hidden), torch.ones(width, dtype=BF16, device=device), matrix(vocab, width))


def to_e4m3_rows(w: torch.Tensor):
    """E4M3 codes and a scale per row of a weight matrix (done once, when the weights are loaded). A row of zeros has
    scale 0 and codes 0."""
    scale = w.float().abs().amax(1) / 448
    safe = torch.where(scale > 0, scale, 1.0)
    return (w.float() / safe[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), scale


def add_product(h: torch.Tensor, w: torch.Tensor, residual: torch.Tensor) -> torch.Tensor:
    """residual + h w^T, the addition in the product's epilogue; `residual` is overwritten."""
    M, K = h.shape
    g.gemm_bf16_fused(h, w, residual, M, w.shape[0], K, g.epilogue(beta=1.0))
    return residual


def serve(attention, stream, w: Weights, gate8, up8, top: int = 8, temperature: float = 1.0):
    """One decoding step after the attention's output: (chosen tokens, their log probabilities, alternatives)."""
    n = g.rms_norm(attention, w.norm, residual=stream, out="e4m3")
    h = g.glu_e4m3(n.y, n.scales, *gate8, *up8)
    stream = add_product(h, w.down, n.sum)
    logits = g.matmul_bf16(g.rms_norm(stream, w.final_norm).y, w.head)
    r = g.token_logprobs(logits, top=top, scale=1.0 / temperature)
    return r.top_ids[:, 0], r.top_logprobs[:, 0], r


def transposed_product(a: torch.Tensor, b: torch.Tensor) -> torch.Tensor:
    """a^T b for BF16 a (rows x m), b (rows x n): the product takes its operands with the summed dimension innermost
    and a multiple of 8 (zeros add nothing)."""
    pad = (0, -a.shape[0] % 8)
    return g.matmul_bf16(torch.nn.functional.pad(a.t(), pad).contiguous(),
                         torch.nn.functional.pad(b.t(), pad).contiguous())


def train_step(attention, stream, tokens, w: Weights, entropy_weight: float = 0.01):
    """(objective per row, gradient of its sum for each weight, gradient of the residual stream)."""
    n1 = g.rms_norm(attention, w.norm, residual=stream, save=True)
    h, saved = g.glu_bf16(n1.y, w.gate, w.up, save=True)
    out = add_product(h, w.down, n1.sum.clone())
    n2 = g.rms_norm(out, w.final_norm, save=True)
    logits = g.matmul_bf16(n2.y, w.head)
    r = g.token_logprobs(logits, tokens)
    objective = r.logprob + entropy_weight * r.entropy

    ones = torch.ones_like(r.logprob)
    dlogits = g.token_logprobs_backward(logits, tokens, r.lse, r.entropy, ones, entropy_weight * ones, inplace=True)
    dy2 = g.matmul_bf16(dlogits, w.head.t().contiguous())
    dhead = transposed_product(dlogits, n2.y)
    dout, dfinal = g.rms_norm_backward(dy2, n2.sum, w.final_norm, n2.rstd)
    dh = g.matmul_bf16(dout, w.down.t().contiguous())
    ddown = transposed_product(dout, h)
    dy1, dgate, dup = g.glu_bf16_backward(dh, n1.y, w.gate, w.up, saved)
    dstream, dnorm = g.rms_norm_backward(dy1, n1.sum, w.norm, n1.rstd, dsum=dout)
    return objective, Weights(dnorm, dgate, dup, ddown, dfinal, dhead), dstream


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rows", type=int, default=64)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=2816)
    ap.add_argument("--vocab", type=int, default=32000)
    a = ap.parse_args()
    w = random_weights(a.width, a.hidden, a.vocab)
    gen = torch.Generator(device="cuda").manual_seed(1)
    attention, stream = (torch.randn(a.rows, a.width, generator=gen, device="cuda").to(BF16) for _ in range(2))
    tokens, logprob, r = serve(attention, stream, w, to_e4m3_rows(w.gate), to_e4m3_rows(w.up))
    print(f"served {a.rows} rows: first tokens {tokens[:4].tolist()}, log probabilities "
          f"{[round(v, 3) for v in logprob[:4].tolist()]}, mean entropy {r.entropy.mean().item():.3f}")
    objective, grads, _ = train_step(attention, stream, tokens.long(), w)
    print(f"mean objective {objective.mean().item():.4f}; gradient norms "
          + ", ".join(f"{k} {v.float().norm().item():.3g}" for k, v in grads._asdict().items()))


if __name__ == "__main__":
    main()
