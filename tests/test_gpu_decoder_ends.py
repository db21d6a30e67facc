"""The operators at a decoder's ends together (examples/decoder_ends.py), on other streams than the current one, and on
several at once.

The step rounds to BF16 between the operators (six times on the way to a gradient: the lookup, two norms' outputs, the
logits' gradient and two norms' gradients, 2^-8 relative each at most, and the table's twice more), so gradients agree in
norm within 8 x 2^-8. A loss moves by what the roundings of the stream before the head (2^-8 of each of its values, 2.5 of
them) leave of a logit: the logits are sums of `width` products of about 1 with weights of 1 / sqrt(width), so in the mean
over their signs 2.5 x 2^-8 x 1, of which 8 standard deviations are 0.08.
"""
import importlib.util
import os

import pytest
import torch

import dense_tensor_core_persistent_gb300 as g
from dense_tensor_core_persistent_gb300 import build as gbuild

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16
A_WHILE = 100_000_000  # clock cycles, some 50 ms
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_ends.py")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gbuild.build()


@pytest.fixture(scope="module")
def ends(_built):
    spec = importlib.util.spec_from_file_location("decoder_ends", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def chain(tokens, w, width):
    def norm(x, weight, bias):
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        return (x - mean) / (var + 1e-5).sqrt() * weight + bias

    x = w["table"][tokens.clamp(min=0)] * width ** 0.5 * (tokens >= 0)[:, None]
    x = norm(norm(x, w["first_weight"], w["first_bias"]), w["last_weight"], w["last_bias"])
    return x @ w["table"].T


@pytest.mark.parametrize("rows,width,vocab", [(1, 64, 300), (37, 264, 2001), (700, 512, 5003)])
def test_steps(ends, rows, width, vocab):
    w = ends.random_weights(width, vocab, seed=rows)
    gen = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.randint(0, vocab, (rows + 1,), generator=gen, device="cuda")
    tokens, targets = ids[:-1].clone(), ids[1:].clone()
    if rows > 8:
        tokens[3], targets[5], targets[6] = -1, -1, -7
        tokens[10:20] = tokens[9]  # a frequent token
    loss, grads = ends.train_step(tokens, targets, w, z_loss=1e-3)

    wd = {k: v.double().requires_grad_() for k, v in w._asdict().items()}
    z = chain(tokens, wd, width)
    lse = torch.logsumexp(z, 1)
    given = targets >= 0
    want = (lse - z.gather(1, targets.clamp(min=0)[:, None])[:, 0]) * given
    ((want + 1e-3 * lse ** 2 * given).sum() / given.sum()).backward()
    assert (loss.double() - want).abs().max() <= 0.08 and torch.all(loss[~given] == 0)
    for k, v in grads._asdict().items():
        ref = wd[k].grad
        assert v.shape == ref.shape and v.isfinite().all()
        assert (v.double() - ref).norm() <= 8 * 2.0 ** -8 * ref.norm(), k
    assert (ends.score(tokens, targets, w).double() + want).abs().max() <= 0.08


def test_step_captured_beside_an_eager_one(ends):
    """One captured step replayed on new tokens while the same weights take eager steps on another stream."""
    w = ends.random_weights(256, 3001)
    gen = torch.Generator(device="cuda").manual_seed(4)
    a, b = (torch.randint(0, 3001, (901,), generator=gen, device="cuda") for _ in range(2))
    want_a, want_b = ends.train_step(a[:-1], a[1:], w), ends.train_step(b[:-1], b[1:], w)
    tokens, targets = a[:-1].clone(), a[1:].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ends.train_step(tokens, targets, w)
    tokens.copy_(b[:-1])
    targets.copy_(b[1:])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        graph.replay()
        with torch.cuda.stream(side):
            eager = ends.train_step(a[:-1], a[1:], w)
    torch.cuda.synchronize()
    for (loss, grads), (want, want_grads) in ((got, want_b), (eager, want_a)):
        assert torch.equal(loss, want) and all(torch.equal(u, v) for u, v in zip(grads, want_grads))


# ---------------------------------------------------------------- memory on another stream than the current one

NAMES = ["layer_norm", "layer_norm_e4m3", "layer_norm_backward", "embedding", "embedding_backward", "embedding_backward_base",
         "embedding_backward_few", "cross_entropy", "cross_entropy_few", "cross_entropy_backward"]


def operator(name):
    """(a call, the tensors it takes)."""
    gen = torch.Generator(device=DEV).manual_seed(len(name))

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV).to(BF16)

    if name.startswith("layer_norm"):
        x, r, w, b = normal(2000, 1024), normal(2000, 1024), normal(1024), normal(1024)
        if name != "layer_norm_backward":
            out = "e4m3" if name.endswith("e4m3") else "bf16"
            return (lambda x, w, b, r, stream=None: g.layer_norm(x, w, b, residual=r, out=out, save=True, stream=stream),
                    [x, w, b, r])
        n = g.layer_norm(x, w, b, residual=r, save=True)
        return g.layer_norm_backward, [normal(2000, 1024), n.sum, w, n.mean, n.rstd, r]
    if name.startswith("embedding"):
        rows = 100 if name.endswith("few") else 3000
        tokens = torch.randint(-1, 500, (rows,), generator=gen, device=DEV)
        if name == "embedding":
            return g.embedding, [normal(500, 1024), tokens]
        if name.endswith("base"):
            return (lambda dy, t, base, stream=None: g.embedding_backward(dy, t, 500, base=base, stream=stream),
                    [normal(rows, 1024), tokens, normal(500, 1024)])
        return lambda dy, t, stream=None: g.embedding_backward(dy, t, 500, stream=stream), [normal(rows, 1024), tokens]
    rows = 20 if name.endswith("few") else 300
    x, head, targets = normal(rows, 512), normal(4000, 512), torch.randint(-1, 4000, (rows,), generator=gen, device=DEV)
    if name != "cross_entropy_backward":
        return g.cross_entropy, [x, head, targets]
    r = g.cross_entropy(x, head, targets)
    return (lambda x, head, t, lse, dloss, stream=None: g.cross_entropy_backward(x, head, t, lse, dloss,
                                                                                 workspace=2 * 300 * 1024, stream=stream),
            [x, head, targets, r.lse, torch.ones(rows, device=DEV)])


def tensors(got):
    return [got] if isinstance(got, torch.Tensor) else [t for t in got if t is not None]


def bits(t):
    return t.contiguous().view(torch.uint8)


def same(a, b):
    return all(torch.equal(bits(x), bits(y)) for x, y in zip(tensors(a), tensors(b)))


def fill_the_like(ts):
    """Takes memory of the sizes of `ts` from the current stream and gives it back with writes still to come."""
    for t in [torch.empty_like(t) for t in ts for _ in range(2)]:
        bits(t).fill_(0xFF)


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_outputs_do_not_take_memory_that_the_current_stream_still_writes(name, handle):
    call, args = operator(name)
    want = call(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(A_WHILE)
    fill_the_like(tensors(want))
    got = call(*args, stream=side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_inputs_are_kept_until_the_other_stream_has_read_them(name):
    call, args = operator(name)
    want = call(*args)
    sizes = [torch.empty_like(t, device="meta") for t in args]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(A_WHILE)
    got = call(*args, stream=side)
    del args
    fill_the_like([torch.empty_like(t, device=DEV) for t in sizes])
    torch.cuda.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_kept_until_the_current_stream_has_read_them(name):
    call, args = operator(name)
    want = call(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(*args, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(A_WHILE)
    copies = [t.clone() for t in tensors(got)]
    del got
    with torch.cuda.stream(side):
        fill_the_like(copies)
    torch.cuda.synchronize()
    assert same(copies, want)


@pytest.mark.parametrize("name", NAMES)
def test_a_call_waits_for_what_the_stream_did_before_it(name):
    """Inputs that a slow kernel of the same stream has yet to write, and outputs that one has yet to read: a launch that
    starts before the one ahead of it ends must not touch memory early."""
    call, args = operator(name)
    want = call(*args)
    late = [torch.zeros_like(t) for t in args]
    torch.cuda.synchronize()
    torch.cuda._sleep(A_WHILE)
    for t, v in zip(late, args):
        t.copy_(v)
    got = call(*late)
    for t in late:  # and what follows must not overtake it
        t.zero_()
    torch.cuda.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_two_calls_at_once_on_two_streams(name):
    call, args = operator(name)
    want = call(*args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(call(*args))
    torch.cuda.synchronize()
    assert all(same(v, want) for v in got)
