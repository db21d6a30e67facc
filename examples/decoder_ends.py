"""The two ends of a decoder with tied weights from the library's operators, as a training step and as a serving step.

    token ids -> embedding (scaled) -> layer norm -> [the decoder's blocks] -> layer norm -> head (the same table) -> loss

`train_step` returns the loss of each position and the gradient of every weight; the table's is the head's with the
lookup's added to it, and no array of rows x vocabulary logits is stored. `score` gives the log probabilities of given
tokens. The blocks are a function and its gradient (the identity here: examples/feed_forward.py has a block). Run it on a
GPU:

    python examples/decoder_ends.py --rows 512 --width 1024 --vocab 32000
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
    """table: vocab x width, the embedding and the head; the norms' weights and biases: width (all BF16)."""
    table: torch.Tensor
    first_weight: torch.Tensor
    first_bias: torch.Tensor
    last_weight: torch.Tensor
    last_bias: torch.Tensor


def random_weights(width: int, vocab: int, device="cuda", seed: int = 0) -> Weights:
    gen = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(*shape, generator=gen, device=device) * std).to(BF16)

    return Weights(normal(vocab, width, std=width ** -0.5), 1 + normal(width, std=0.1), normal(width, std=0.1),
                   1 + normal(width, std=0.1), normal(width, std=0.1))


def forward(tokens, w: Weights, save: bool):
    """The stream before the head, and what its gradient needs."""
    scale = w.table.shape[1] ** 0.5
    first = g.layer_norm(g.embedding(w.table, tokens, scale=scale), w.first_weight, w.first_bias, save=save)
    return first, g.layer_norm(first.y, w.last_weight, w.last_bias, save=save)


def score(tokens, targets, w: Weights):
    """Log probabilities of `targets` (negative: none, 0)."""
    return -g.cross_entropy(forward(tokens, w, save=False)[1].y, w.table, targets).loss


def train_step(tokens, targets, w: Weights, z_loss: float = 1e-4):
    """(loss of each position, gradient of their mean plus z_loss * the mean of lse^2 for each weight)."""
    first, last = forward(tokens, w, save=True)
    r = g.cross_entropy(last.y, w.table, targets)
    given = (targets >= 0).float()
    share = given / given.sum().clamp(min=1.0)
    dlast, dtable = g.cross_entropy_backward(last.y, w.table, targets, r.lse, share, dlse=2 * z_loss * r.lse * share)
    dfirst, *dlast_affine = g.layer_norm_backward(dlast, last.sum, w.last_weight, last.mean, last.rstd)
    dembedded, *dfirst_affine = g.layer_norm_backward(dfirst, first.sum, w.first_weight, first.mean, first.rstd)
    vocab, width = w.table.shape
    g.embedding_backward(dembedded, tokens, vocab, scale=width ** 0.5, base=dtable, inplace=True)
    return r.loss, Weights(dtable, *dfirst_affine, *dlast_affine)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rows", type=int, default=512)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--vocab", type=int, default=32000)
    a = ap.parse_args()
    w = random_weights(a.width, a.vocab)
    gen = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, a.vocab, (a.rows + 1,), generator=gen, device="cuda")
    loss, grads = train_step(ids[:-1], ids[1:], w)
    print(f"mean loss {loss.mean().item():.4f}; gradient norms "
          + ", ".join(f"{k} {v.float().norm().item():.3g}" for k, v in grads._asdict().items()))
    print(f"first log probabilities {[round(v, 3) for v in score(ids[:-1], ids[1:], w)[:4].tolist()]}")


if __name__ == "__main__":
    main()
