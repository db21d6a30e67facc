"""gemm_token_logprobs and its gradient through the binding, against FP64 evaluations of their definitions.

Tolerances, derived before the first run, with u = 2^-24. A thread adds at most n = ceil(vocab / 512) + 8
terms one after another and the partial sums join in a tree, each exp being within 2^-22 of its value plus
the rounding of its argument (weighted by the exp itself, x e^-x < 1): the sum of exponentials has a
relative error below d = (n + 64) 2 u. lse and the log probabilities then carry d and the roundings of the
numbers they are made of; the entropy carries d times the size of its two terms; a probability computed
from the FP32 lse carries lse's error as a relative one.
"""
import math

import pytest
import torch

import dense_tensor_core_persistent_gb300 as g
from dense_tensor_core_persistent_gb300 import build as gbuild

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gbuild.build()


def problem(rows, vocab, dtype, seed, spread=3.0):
    gen = torch.Generator().manual_seed(seed)
    l = (torch.randn(rows, vocab, generator=gen) * spread).to(dtype)
    t = torch.randint(0, vocab, (rows,), generator=gen)
    if rows > 2:
        t[1] = -1
    return l, t


def delta(vocab):
    return (math.ceil(vocab / 512) + 72) * 2 * U


def definition(l, t, scale=1.0):
    z = l.double() * scale
    lse = torch.logsumexp(z, 1)
    logp = z - lse[:, None]
    p = logp.exp()
    ent = -torch.where(p > 0, p * logp, 0.0).sum(1)
    lp = torch.where(t >= 0, logp.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
    return lse, logp, p, ent, lp


def check(l, t, scale=1.0, top=0, out=None):
    vocab = l.shape[1]
    r = out if out is not None else g.token_logprobs(l.to(DEV), t.to(DEV), top=top, scale=scale)
    lse, logp, p, ent, lp = definition(l, t, scale)
    d = delta(vocab)
    size = lse.abs() + math.log(vocab) + (l.double() * scale).amax(1).abs()
    tol = d + 8 * U * size
    assert torch.all((r.lse.cpu().double() - lse).abs() <= tol)
    assert torch.all((r.logprob.cpu().double() - lp).abs() <= tol + 8 * U * lp.abs())
    assert torch.all((r.entropy.cpu().double() - ent).abs() <= 4 * d * (1 + math.log(vocab)))
    if top:
        order = torch.sort(l.float() + 0.0, dim=1, descending=True, stable=True).indices[:, :top]
        assert torch.equal(r.top_ids.cpu().long(), order)
        want = logp.gather(1, order)
        assert torch.all((r.top_logprobs.cpu().double() - want).abs() <= tol[:, None] + 8 * U * want.abs())
    return r


SHAPES = [(1, 1), (1, 7), (1, 8), (3, 1000), (2, 131072), (5, 50001), (400, 257), (3, 9001), (700, 4104), (2, 262147)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("top", [0, 1, 20])
def test_forward(rows, vocab, dtype, top):
    l, t = problem(rows, vocab, dtype, rows * 7 + vocab)
    check(l, t, top=min(top, vocab))
    check(l, t, scale=0.7, top=min(top, vocab))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(3, 5000), (350, 3001), (1, 131072)])
def test_ties_go_to_the_lower_index(rows, vocab, dtype):
    gen = torch.Generator().manual_seed(vocab)
    l = torch.randint(-3, 3, (rows, vocab), generator=gen).to(dtype)
    l[l == 0] *= -1.0  # -0 and 0 are equal
    l[0, :] = 1.0
    check(l, torch.zeros(rows, dtype=torch.int64), top=32)


@pytest.mark.parametrize("dtype", TYPES)
def test_many_candidates_in_few_threads(dtype):
    """Large logits wherever 20 threads read: more candidates than the list holds."""
    n = 8 if dtype == torch.bfloat16 else 4
    vocab = 8 * 512 * n * 16
    gen = torch.Generator().manual_seed(3)
    l = torch.rand(1, vocab, generator=gen)
    owner = (torch.arange(vocab) // n) % 512
    l[:, owner < 20] += 8 * torch.rand(1, int((owner < 20).sum()), generator=gen) + 2
    check(l.to(dtype), torch.tensor([5]), top=20)
    check(l.to(dtype), torch.tensor([5]), top=32)


@pytest.mark.parametrize("dtype", TYPES)
def test_masked_logits(dtype):
    rows, vocab = 9, 3003
    l, t = problem(rows, vocab, dtype, 5)
    lowest = torch.finfo(dtype).min
    keep = l.clone()
    l[0, 1:] = -math.inf           # one logit left
    l[1, :-1] = -math.inf
    l[2] = -math.inf               # nothing left
    l[3, ::2] = -math.inf
    l[4, 5:] = lowest              # the lowest value next to ordinary ones
    l[5] = lowest                  # everywhere: uniform
    l[6, 1500:] = -math.inf
    t = torch.tensor([0, vocab - 1, 4, 1, 2, 7, 1501, -1, 3])
    r = g.token_logprobs(l.to(DEV), t.to(DEV), top=5)
    lse, ent, lp = (x.cpu() for x in (r.lse, r.entropy, r.logprob))
    assert lp[0] == 0 and ent[0] == 0 and lse[0] == keep[0, 0].float()
    assert lp[1] == 0 and ent[1] == 0
    assert lse[2] == -math.inf and ent[2] == 0 and lp[2] == -math.inf
    assert r.top_ids[2].tolist() == [0, 1, 2, 3, 4] and torch.all(r.top_logprobs[2].cpu() == -math.inf)
    assert abs(lp[5].item() + math.log(vocab)) <= 1e-5 and abs(ent[5].item() - math.log(vocab)) <= 1e-4
    assert lp[6] == -math.inf and torch.isfinite(ent[6])
    assert r.top_ids[0].tolist() == [0, 1, 2, 3, 4] and r.top_ids[1].tolist() == [vocab - 1, 0, 1, 2, 3]
    for i in (3, 4, 6, 7, 8):
        _, logp, p, e, want = definition(l[i:i + 1], t[i:i + 1])
        assert abs(ent[i].item() - e.item()) <= 4 * delta(vocab) * 9
        assert want.item() == lp[i].item() or abs(want.item() - lp[i].item()) <= delta(vocab) + 1e-5
    # gradients: zero at masked places, nothing from the empty row
    dlp, dh = torch.ones(rows), torch.full((rows,), 0.3)
    dl = g.token_logprobs_backward(l.to(DEV), t.to(DEV), r.lse, r.entropy, dlp.to(DEV), dh.to(DEV)).cpu()
    assert torch.isfinite(dl[[0, 1, 2, 3, 4, 5, 7, 8]]).all()
    assert torch.all(dl[2] == 0) and torch.all(dl[3, ::2] == 0) and torch.all(dl[0, 1:] == 0)


@pytest.mark.parametrize("dtype", TYPES)
def test_nan_infinity_and_tokens_outside(dtype):
    rows, vocab = 5, 2001
    l, _ = problem(rows, vocab, dtype, 8)
    l[0, 77] = math.nan
    l[0, 1900] = math.nan
    l[1, 5] = math.inf
    t = torch.tensor([3, 4, vocab, -5, vocab - 1])
    r = g.token_logprobs(l.to(DEV), t.to(DEV), top=3)
    lp = r.logprob.cpu()
    assert r.lse[0].isnan() and lp[0].isnan() and r.entropy[0].isnan() and lp[1].isnan()
    assert r.top_ids[0].tolist()[:2] == [77, 1900] and r.top_ids[1].tolist()[0] == 5
    assert lp[2].isnan() and lp[3] == 0 and lp[4].isfinite() and r.lse[2].isfinite()
    dl = g.token_logprobs_backward(l.to(DEV), t.to(DEV), r.lse, r.entropy, torch.ones(rows, device=DEV)).cpu()
    assert dl[2].isnan().all() and dl[0].isnan().all()
    assert torch.all(dl[3] == 0) and dl[4].isfinite().all()


@pytest.mark.parametrize("dtype", TYPES)
def test_strided_rows_at_any_alignment(dtype):
    rows, vocab = 6, 1021
    for off, ld in ((0, 1021), (1, 1030), (3, 1024), (5, 1037)):
        l, t = problem(rows, vocab, dtype, off + ld)
        wide = torch.full((rows, ld + 8), 50.0, dtype=dtype, device=DEV)
        view = wide[:, off:off + vocab]
        view.copy_(l)
        r = g.token_logprobs(view, t.to(DEV), top=7)
        check(l, t, top=7, out=r)
        dlp, dh = torch.randn(rows), torch.randn(rows)
        dl = g.token_logprobs_backward(view, t.to(DEV), r.lse, r.entropy, dlp.to(DEV), dh.to(DEV))
        again = g.token_logprobs_backward(view, t.to(DEV), r.lse, r.entropy, dlp.to(DEV), dh.to(DEV), inplace=True)
        assert again.data_ptr() == view.data_ptr() and torch.equal(view, dl)
        outside = torch.ones(ld + 8, dtype=torch.bool, device=DEV)
        outside[off:off + vocab] = False
        assert torch.all(wide[:, outside] == 50.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_backward(rows, vocab, dtype):
    scale = 0.9
    l, t = problem(rows, vocab, dtype, rows + 3 * vocab)
    gen = torch.Generator().manual_seed(1)
    dlp, dh = torch.randn(rows, generator=gen), torch.randn(rows, generator=gen)
    r = g.token_logprobs(l.to(DEV), t.to(DEV), scale=scale)
    _, logp, p, ent, _ = definition(l, t, scale)
    size = logp.abs() + math.log(vocab) + (l.double() * scale).abs().amax(1, keepdim=True)
    rel = 4 * delta(vocab) + 32 * U * size
    half = 2.0 ** -8 if dtype == torch.bfloat16 else U
    for use_lp, use_h in ((True, True), (True, False), (False, True)):
        a = torch.where(t >= 0, dlp, 0.0).double()[:, None] if use_lp else torch.zeros(rows, 1, dtype=torch.float64)
        b = dh.double()[:, None] if use_h else torch.zeros(rows, 1, dtype=torch.float64)
        hot = torch.zeros_like(p).scatter_(1, t.clamp(min=0)[:, None], 1.0)
        want = scale * (a * (hot - p) - b * p * (logp + ent[:, None]))
        terms = scale * (a.abs() * (hot + p) + b.abs() * p * (logp.abs() + ent[:, None] + 4 * math.log(vocab + 1)))
        got = g.token_logprobs_backward(l.to(DEV), t.to(DEV) if use_lp else None, r.lse, r.entropy,
                                        dlp.to(DEV) if use_lp else None, dh.to(DEV) if use_h else None, scale=scale)
        assert got.dtype == dtype
        assert torch.all((got.cpu().double() - want).abs() <= half * want.abs() + rel * terms + 1e-37)


def test_backward_against_differences():
    rows, vocab, scale = 2, 12, 1.3
    l, t = problem(rows, vocab, torch.float32, 9)
    dlp, dh = torch.tensor([0.7, -1.1]), torch.tensor([0.4, 0.2])
    r = g.token_logprobs(l.to(DEV), t.to(DEV), scale=scale)
    dl = g.token_logprobs_backward(l.to(DEV), t.to(DEV), r.lse, r.entropy, dlp.to(DEV), dh.to(DEV), scale=scale).cpu()

    def value(x):
        _, _, _, ent, lp = definition(x, t, scale)
        return (dlp.double() * lp + dh.double() * ent).sum().item()

    h = 1e-5
    for i in range(rows):
        for j in range(vocab):
            e = torch.zeros(rows, vocab, dtype=torch.float64)
            e[i, j] = h
            diff = (value(l.double() + e) - value(l.double() - e)) / (2 * h)
            assert abs(dl[i, j].item() - diff) <= 2e-6 * (1 + abs(diff))


def test_repeats_stream_graph_and_empty():
    l, t = problem(64, 30001, torch.bfloat16, 12)
    ld, td = l.to(DEV), t.to(DEV)
    dlp = torch.ones(64, device=DEV)
    want = g.token_logprobs(ld, td, top=8)
    dwant = g.token_logprobs_backward(ld, td, want.lse, want.entropy, dlp)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = g.token_logprobs(ld, td, top=8, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = g.token_logprobs(ld, td, top=8)
        d = g.token_logprobs_backward(ld, td, r.lse, r.entropy, dlp)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(r, want)) and torch.equal(d, dwant)
    none = g.token_logprobs(ld[:0], td[:0], top=8)
    assert none.lse.numel() == 0 and none.top_ids.shape == (0, 8)
    free = g.token_logprobs(ld)
    assert free.logprob is None and torch.equal(free.lse, want.lse)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("others", [-44.0, -4.0])
def test_rows_that_one_logit_dominates(dtype, others):
    """A largest logit of 16, one of 16 - `lag` read by the same thread, in the same chunk of a row or in an earlier one,
    and others far below: small log probabilities and entropies keep their digits and their signs.

    Each power of two carries the rounding of an argument below 2^7 and its own, 1e-5 of itself with a margin; next to the
    maximum, up to 64 of the other 70000 may be rounded off."""
    rows, vocab = 320, 70000
    n = 8 if dtype == torch.bfloat16 else 4
    l = torch.full((rows, vocab), others)
    t = torch.zeros(rows, dtype=torch.int64)
    for i in range(rows):
        lag, chunk, u, owner = (0.5, 3.0, 6.0, 8.0, 10.875)[i % 5], (0, 1, 3)[i // 5 % 3], i // 15 % 3, 37 * i % 256
        first, later = n * owner, n * (owner + 256 * u + 2048 * chunk)
        l[i, first + i % n] = 16.0 - lag
        l[i, later + (i + 3) % n] = 16.0
        t[i] = later + (i + 3) % n
    l, t = l.to(dtype).to(DEV), t.to(DEV)
    r = g.token_logprobs(l, t, top=2)
    z = l.double()
    rest = torch.exp(z - 16.0).sum(1) - 1.0
    lp = -torch.log1p(rest)
    p = torch.exp(z - 16.0 + lp[:, None])
    ent = -(p * (z - 16.0 + lp[:, None])).sum(1)
    rel = 1e-5 + 64 / 70000
    assert torch.all(r.logprob <= 0) and torch.all(r.entropy >= 0)
    assert torch.all((r.logprob.double() - lp).abs() <= rel * lp.abs())
    assert torch.all((r.entropy.double() - ent).abs() <= rel * ent)
    assert torch.equal(r.top_logprobs[:, 0], r.logprob) and torch.equal(r.top_ids[:, 0].long(), t)
    assert torch.all((r.lse.double() - 16.0 + lp).abs() <= 32 * U)


@pytest.mark.parametrize("dtype", TYPES)
def test_nan_at_the_first_index_among_many_candidates(dtype):
    """More candidates than the list holds, the first logit NaN: it still comes first."""
    l = torch.ones(3, 5001)
    l[0] = math.nan
    l[1, 0] = math.nan
    l[1, 4000] = math.nan
    r = g.token_logprobs(l.to(dtype).to(DEV), top=3)
    assert r.top_ids.tolist() == [[0, 1, 2], [0, 4000, 1], [0, 1, 2]]
    assert r.lse[:2].isnan().all() and r.lse[2].isfinite()


@pytest.mark.parametrize("dtype", TYPES)
def test_large_gradients_leave_masked_logits_alone(dtype):
    """Gradients of the entropy as large as a loss scale makes them: masked logits still get 0."""
    l, t = problem(3, 1000, dtype, 4)
    l[:, ::3] = -math.inf
    l[:, 1::3] = torch.finfo(dtype).min
    t = torch.tensor([2, 5, 8])
    r = g.token_logprobs(l.to(DEV), t.to(DEV))
    dl = g.token_logprobs_backward(l.to(DEV), t.to(DEV), r.lse, r.entropy, torch.ones(3, device=DEV),
                                   torch.tensor([1e9, -1e12, 1e30], device=DEV)).cpu()
    assert torch.all(dl[:, ::3] == 0) and torch.all(dl[:, 1::3] == 0)
    assert dl.isfinite().all() and torch.all(dl[:, 2] != 0)


@pytest.mark.parametrize("dtype", TYPES)
def test_token_outside_in_a_row_of_nothing(dtype):
    """A token past the vocabulary makes its row NaN, also where the row has no mass."""
    l = torch.full((3, 77), -math.inf, dtype=dtype, device=DEV)
    t = torch.tensor([77, 3, -1], device=DEV)
    r = g.token_logprobs(l, t)
    assert r.logprob[0].isnan() and r.logprob[1] == -math.inf and r.logprob[2] == 0
    dl = g.token_logprobs_backward(l, t, r.lse, r.entropy, torch.ones(3, device=DEV), torch.ones(3, device=DEV))
    assert dl[0].isnan().all() and torch.all(dl[1:] == 0)


def test_missing_tensors_are_refused():
    l = torch.zeros(2, 32, dtype=torch.bfloat16, device=DEV)
    one = torch.ones(2, device=DEV)
    for call in (lambda: g.token_logprobs_backward(l, None, None, None, None),
                 lambda: g.rms_norm(None),
                 lambda: g.rms_norm_backward(l, l, None, None),
                 lambda: g.rms_norm_backward(None, l, None, one),
                 lambda: g.glu_bf16_backward(l, l, torch.zeros(32, 32, dtype=torch.bfloat16, device=DEV),
                                             torch.zeros(32, 32, dtype=torch.bfloat16, device=DEV), None)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("rows,vocab,dtype", [(153, 262147, torch.float32), (153, 524293, torch.bfloat16)])
def test_several_rows_a_cluster(rows, vocab, dtype):
    """More rows than clusters of CTAs that share one, each with alternatives."""
    gen = torch.Generator(device=DEV).manual_seed(vocab)
    l = torch.randn(rows, vocab, generator=gen, device=DEV)
    l = (l * (0.5 + 3 * torch.rand(rows, 1, generator=gen, device=DEV))).to(dtype)
    t = torch.randint(0, vocab, (rows,), generator=gen, device=DEV)
    r = g.token_logprobs(l, t, top=20)
    lse, logp, _, ent, lp = definition(l, t)
    d = delta(vocab)
    tol = d + 8 * U * (lse.abs() + math.log(vocab) + l.double().amax(1).abs())
    assert torch.all((r.lse.double() - lse).abs() <= tol)
    assert torch.all((r.logprob.double() - lp).abs() <= tol + 8 * U * lp.abs())
    assert torch.all((r.entropy.double() - ent).abs() <= 4 * d * (1 + math.log(vocab)))
    order = torch.sort(l.float() + 0.0, dim=1, descending=True, stable=True).indices[:, :20]
    assert torch.equal(r.top_ids.long(), order)
    want = logp.gather(1, order)
    assert torch.all((r.top_logprobs.double() - want).abs() <= tol[:, None] + 8 * U * want.abs())
    again = g.token_logprobs(l, t, top=20)
    assert all(torch.equal(a, b) for a, b in zip(r, again))
