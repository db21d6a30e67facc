"""examples/feed_forward.py: the serving and the training step against FP64 (autograd for the gradients).

The step rounds to BF16 between the operators (about eight times on the way to a gradient, 2^-8 relative each, at
most), so gradients agree in norm within 8 x 2^-8, and log probabilities within what one BF16 rounding of logits of
the size seen here and the roundings before it leave. The E4M3 step adds a 2^-4 relative rounding of each operand of two products
of the block, which average over the summed dimension: its log probabilities are compared with the BF16 chain's scale.
"""
import importlib.util
import os

import pytest
import torch

from dense_tensor_core_persistent_gb300 import build as gbuild

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward.py")


@pytest.fixture(scope="module")
def ff():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gbuild.build()
    spec = importlib.util.spec_from_file_location("feed_forward", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def chain(w, attention, stream):
    def norm(x, weight):
        return x / (x.square().mean(1, keepdim=True) + 1e-5).sqrt() * weight

    s = attention + stream
    y = norm(s, w["norm"])
    h = torch.nn.functional.silu(y @ w["gate"].T) * (y @ w["up"].T)
    out = s + h @ w["down"].T
    return torch.log_softmax(norm(out, w["final_norm"]) @ w["head"].T, 1)


@pytest.mark.parametrize("rows,width,hidden,vocab", [(8, 256, 512, 1000), (37, 264, 520, 2008)])
def test_steps(ff, rows, width, hidden, vocab):
    w = ff.random_weights(width, hidden, vocab, seed=rows)
    gen = torch.Generator(device="cuda").manual_seed(2)
    attention, stream = (torch.randn(rows, width, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    tokens = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    objective, grads, dstream = ff.train_step(attention, stream, tokens, w, entropy_weight=0.1)

    wd = {k: v.double().requires_grad_() for k, v in w._asdict().items()}
    sd = stream.double().requires_grad_()
    logp = chain(wd, attention.double(), sd)
    entropy = -(logp.exp() * logp).sum(1)
    want = logp.gather(1, tokens[:, None])[:, 0] + 0.1 * entropy
    want.sum().backward()
    assert (objective.double() - want).abs().max() <= 0.06
    for k, v in grads._asdict().items():
        ref = wd[k].grad
        assert v.shape == ref.shape
        assert (v.double() - ref).norm() <= 8 * 2.0 ** -8 * ref.norm(), k
    assert (dstream.double() - sd.grad).norm() <= 8 * 2.0 ** -8 * sd.grad.norm()

    if width % 16 == 0:
        chosen, logprob, r = ff.serve(attention, stream, w, ff.to_e4m3_rows(w.gate), ff.to_e4m3_rows(w.up), top=4)
        at = logp.detach().gather(1, chosen.long()[:, None])[:, 0]
        assert (logprob.double() - at).abs().max() <= 0.5
        assert torch.all(r.top_logprobs[:, 0] >= r.top_logprobs[:, 3])
