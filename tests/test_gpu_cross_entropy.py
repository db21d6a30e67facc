"""gemm_cross_entropy and its gradient through the binding, against FP64 evaluations of their definitions.

Tolerances, derived before the first run.
  Logits. Products of BF16 values are exact in FP32; a tensor-core step adds 16 of them to the accumulator and may cut
  what lies below the accumulator's last place, so a logit is off by at most (K / 16 + 2) 2^-22 of a, the sum of the
  products' magnitudes: E = scale * that, with the row's largest a.
  Forward. lse moves by at most the largest logit error E; exponentials (2^-22 relative), sums (a tree and chunks, fewer
  than 64 roundings in a row) and the log1p add less than 2^-17 of 1, and the last addition 2^-24 of |lse|. loss has
  two logits' errors. Where the logits are exact (small integers) loss carries only the relative errors of its terms.
  Gradient. p is off by e = E + |lse| 2^-23 + 2^-19 relative. G = scale ((dloss + dlse) p - dloss 1[t]) is off by e on
  its first term and 2^-8 of itself from the rounding to BF16; dX adds G's errors times |W|, (V / 16 + 2 + pieces + 8)
  2^-22 of the sum of magnitudes and 2^-8 of itself; dW alike over the rows.
"""
import pytest
import torch

import dense_tensor_core_persistent_gb300 as g
from dense_tensor_core_persistent_gb300 import build as gbuild

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gbuild.build()


def problem(M, V, K, seed, spread=2.0):
    gen = torch.Generator().manual_seed(seed)
    head = (torch.randn(V, K, generator=gen) * spread / max(K, 1) ** 0.5).to(BF16)
    ids = torch.randint(0, V, (M,), generator=gen)
    x = (torch.randn(M, K, generator=gen) + 4 * torch.rand(M, 1, generator=gen) * head[ids].float()).to(BF16)
    targets = torch.where(torch.rand(M, generator=gen) < 0.15, -1 - ids % 3, ids)
    dloss, dlse = torch.rand(M, generator=gen) / M, torch.randn(M, generator=gen) * 0.1 / M
    return [t.to(DEV) for t in (x, head, targets, dloss, dlse)]


class Definition:
    def __init__(self, x, head, targets, scale):
        self.x, self.w, self.t, self.scale = x.double(), head.double(), targets, scale
        K = x.shape[1]
        self.z = scale * (self.x @ self.w.T)
        self.lse = torch.logsumexp(self.z, 1)
        self.given = targets >= 0
        at = targets.clamp(min=0)
        self.onehot = torch.nn.functional.one_hot(at, head.shape[0]).double() * self.given[:, None]
        self.loss = (self.lse - self.z.gather(1, at[:, None])[:, 0]) * self.given
        self.E = scale * (K / 16 + 2) * 2.0 ** -22 * (self.x.abs() @ self.w.abs().T).amax(1)

    def check_forward(self, r):
        tol = self.E + 2.0 ** -17 + 2.0 ** -24 * self.lse.abs()
        assert torch.all((r.lse.double() - self.lse).abs() <= tol)
        if r.loss is not None:
            assert torch.all((r.loss.double() - self.loss).abs() <= 2 * tol)
            assert torch.all(r.loss[~self.given] == 0) and torch.all(r.loss >= 0)

    def check_backward(self, dloss, dlse, dx, dw, pieces=1):
        zero = torch.zeros_like(self.lse)
        dl = zero if dloss is None else dloss.double() * self.given
        a = (dl + (zero if dlse is None else dlse.double()))[:, None] * (self.z - self.lse[:, None]).exp() * self.scale
        G = a - self.scale * dl[:, None] * self.onehot
        e = (self.E + self.lse.abs() * 2.0 ** -23 + 2.0 ** -19)[:, None]
        dG = e * a.abs() + 2.0 ** -8 * (G.abs() + e * a.abs())
        for got, A, dA, B in ((dx, G, dG, self.w), (dw, G.T, dG.T, self.x)):
            if got is None:
                continue
            want, size = A @ B, A.abs() @ B.abs()
            tol = dA @ B.abs() + (A.shape[1] / 16 + 10 + pieces) * 2.0 ** -22 * size
            assert torch.all((got.double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol) + 1e-37)


# one tile, ragged ones, several waves, both tiles of a CTA pair, tails of a wave as halves
SHAPES = [(1, 1, 8), (2, 3, 16), (1, 131, 64), (5, 257, 72), (33, 1000, 264), (64, 5000, 1032), (129, 8005, 520),
          (300, 513, 128), (257, 130, 2048), (700, 20000, 264), (1025, 9001, 2056), (2100, 5003, 2048)]


@pytest.mark.parametrize("M,V,K", SHAPES)
def test_forward_and_gradient(M, V, K):
    x, head, targets, dloss, dlse = problem(M, V, K, M + V + K)
    r = g.cross_entropy(x, head, targets)
    d = Definition(x, head, targets, 1.0)
    d.check_forward(r)
    dx, dw = g.cross_entropy_backward(x, head, targets, r.lse, dloss, dlse=dlse)
    d.check_backward(dloss, dlse, dx, dw)
    assert g.get_device_status()[0] == 0


@pytest.mark.parametrize("M,V,K", [(1, 700, 64), (40, 3000, 264), (300, 1301, 128), (1025, 5001, 2056)])
@pytest.mark.parametrize("columns", [256, 768])
def test_pieces_of_the_vocabulary(M, V, K, columns):
    x, head, targets, dloss, dlse = problem(M, V, K, 5)
    workspace = 2 * M * columns
    piece = g.cross_entropy_piece(M, V, workspace)
    assert piece <= columns and (piece % 256 == 0 or piece == V)
    r = g.cross_entropy(x, head, targets, scale=0.75)
    d = Definition(x, head, targets, 0.75)
    d.check_forward(r)
    kw = dict(dlse=dlse, scale=0.75, workspace=workspace)
    dx, dw = g.cross_entropy_backward(x, head, targets, r.lse, dloss, **kw)
    d.check_backward(dloss, dlse, dx, dw, pieces=-(-V // piece))
    again = g.cross_entropy_backward(x, head, targets, r.lse, dloss, **kw)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
    only_dx, none = g.cross_entropy_backward(x, head, targets, r.lse, dloss, weight_grad=False, **kw)
    assert none is None
    d.check_backward(dloss, dlse, only_dx, None, pieces=-(-V // piece))
    none, only_dw = g.cross_entropy_backward(x, head, targets, r.lse, dloss, input_grad=False, **kw)
    assert none is None  # (another launch may add the rows in another order)
    d.check_backward(dloss, dlse, None, only_dw)


def test_without_targets_and_without_one_of_the_gradients():
    x, head, targets, dloss, dlse = problem(50, 1003, 136, 8)
    d = Definition(x, head, targets, 1.0)
    r = g.cross_entropy(x, head)
    assert r.loss is None
    d.check_forward(r)
    d.check_backward(None, dlse, *g.cross_entropy_backward(x, head, None, r.lse, None, dlse=dlse))
    d.check_backward(dloss, None, *g.cross_entropy_backward(x, head, targets, r.lse, dloss))


def test_a_row_that_its_target_dominates_keeps_its_digits():
    # integers: every logit is exact; row i's target stands i above 400 others, row 0 ties with one of them
    V, K = 401, 16
    head = torch.zeros(V, K)
    head[:, 0] = -1.0
    head[7, 0] = 0.0
    head[9, 0] = 0.0
    head[9, 1] = -1.0
    x = torch.zeros(40, K)
    x[:, 0] = torch.arange(40.0)
    x[:, 1] = torch.arange(40.0)
    x, head = x.to(BF16).to(DEV), head.to(BF16).to(DEV)
    targets = torch.full((40,), 7, device=DEV)
    r = g.cross_entropy(x, head, targets)
    z = x.double() @ head.double().T
    others = torch.cat([z[:, :7], z[:, 8:]], 1)
    want = torch.log1p((others - z[:, 7:8]).exp().sum(1))
    assert torch.all((r.loss.double() - want).abs() <= 2.0 ** -17 * want)
    assert r.loss[-1] > 0


@pytest.mark.parametrize("V", [255, 256, 257, 5000])
def test_masked_like_columns(V):
    # weights that give logits of about -3e38 and of minus infinity beside ordinary ones, at tile borders too
    gen = torch.Generator().manual_seed(V)
    head = torch.randn(V, 16, generator=gen)
    head[:, 8:] = 0.0
    off = torch.rand(V, generator=gen) < 0.3
    off[0] = False
    off[-1] = True
    head[off, 8] = -3.0e38
    x = torch.randn(6, 16, generator=gen)
    x[:, 8:] = 0.0
    x[:3, 8] = 1.0
    x[3:, 8] = 4.0  # (-1.2e39: minus infinity)
    x, head = x.to(BF16).to(DEV), head.to(BF16).to(DEV)
    targets = torch.zeros(6, dtype=torch.int64, device=DEV)
    r = g.cross_entropy(x, head, targets)
    z = x[:, :8].double() @ head[:, :8].double().T
    z[:, off.to(DEV)] = -torch.inf
    lse = torch.logsumexp(z, 1)
    assert torch.all((r.lse.double() - lse).abs() <= 2.0 ** -16 * (1 + lse.abs()))
    dloss = torch.ones(6, device=DEV)
    dx, dw = g.cross_entropy_backward(x, head, targets, r.lse, dloss)
    p = (z - lse[:, None]).exp()
    p[:, 0] -= 1
    want = p.T @ x.double()
    assert torch.all(dw[off.to(DEV)] == 0)
    assert torch.all((dw.double() - want).abs() <= 2.0 ** -6 * (p.abs().T @ x.double().abs()) + 1e-30)


def test_targets_outside_the_vocabulary_and_rows_of_nan():
    x, head, _, dloss, _ = problem(6, 300, 64, 3)
    targets = torch.tensor([5, 300, -1, 299, 1 << 40, -(1 << 40)], device=DEV)
    x[2] = float("nan")
    x[5, 3] = float("inf")
    r = g.cross_entropy(x, head, targets)
    assert torch.equal(r.loss.isnan().cpu(), torch.tensor([False, True, False, False, True, False]))
    assert r.loss[2] == 0 and r.loss[5] == 0
    assert torch.equal(r.lse.isnan().cpu(), torch.tensor([False, False, True, False, False, True]))
    dx, _ = g.cross_entropy_backward(x, head, targets, r.lse, dloss, weight_grad=False)
    assert torch.equal(dx.isnan().all(1).cpu(), torch.tensor([False, True, False, False, True, False]))
    assert torch.all(dx[2] == 0) and torch.all(dx[5] == 0)  # places without a target, whatever they hold
    assert not dx[0].isnan().any() and not dx[3].isnan().any()


def test_strides_and_what_lies_behind():
    M, V, K = 70, 515, 72
    x, head, targets, dloss, dlse = problem(M, V, K, 21)
    wide = torch.full((M, K + 24), float("nan"), dtype=BF16, device=DEV)
    wide[:, :K] = x
    view = wide[:, :K]
    r, s = g.cross_entropy(view, head, targets), g.cross_entropy(x, head, targets)
    assert torch.equal(r.loss, s.loss) and torch.equal(r.lse, s.lse)
    want = g.cross_entropy_backward(x, head, targets, r.lse, dloss, dlse=dlse)
    got = g.cross_entropy_backward(view, head, targets, r.lse, dloss, dlse=dlse)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    # raw: dX with a stride, and memory around every output
    buf = torch.full((M + 2, K + 8), 7.0, dtype=BF16, device=DEV)
    dw = torch.full((V + 2, K), 7.0, dtype=BF16, device=DEV)
    loss, lse = torch.full((M + 1,), 7.0, device=DEV), torch.full((M + 1,), 7.0, device=DEV)
    g.gemm_cross_entropy(x, head, targets, loss, lse, M, V, K)
    assert loss[M] == 7 and lse[M] == 7 and torch.equal(loss[:M], r.loss)
    for workspace in (0, 2 * M * 256):
        g.gemm_cross_entropy_backward(x, head, targets, lse, dloss, dlse, buf, dw, M, V, K, workspace=workspace,
                                      strides=g.gemm_cross_entropy_strides_t(0, K + 8))
        assert torch.all(buf[M:] == 7) and torch.all(buf[:, K:] == 7) and torch.all(dw[V:] == 7)
        Definition(x, head, targets, 1.0).check_backward(dloss, dlse, buf[:M, :K], dw[:V], pieces=3)
        if workspace == 0:
            assert torch.equal(dw[:V], want[1]) and torch.equal(buf[:M, :K], want[0])


def test_empty():
    x, head, targets, dloss, _ = problem(3, 40, 16, 2)
    none = x[:0]
    r = g.cross_entropy(none, head, targets[:0])
    assert r.loss.shape == (0,) and r.lse.shape == (0,)
    dx, dw = g.cross_entropy_backward(none, head, targets[:0], r.lse, dloss[:0])
    assert dx.shape == (0, 16) and torch.all(dw == 0)
    r = g.cross_entropy(x[:, :0].contiguous(), head[:, :0].contiguous(), targets)
    assert torch.allclose(r.lse, torch.full((3,), 40.0, device=DEV).log(), rtol=2.0 ** -22)
    with pytest.raises(g.GemmError):
        g.cross_entropy(x, head[:0], targets)


def test_gradient_against_differences():
    M, V, K = 4, 300, 64
    x, head, targets, _, _ = problem(M, V, K, 77)
    targets = targets.clamp(min=0)
    dloss, dlse = torch.rand(M, device=DEV), torch.randn(M, device=DEV)
    r = g.cross_entropy(x, head, targets)
    dx, dw = g.cross_entropy_backward(x, head, targets, r.lse, dloss, dlse=dlse)

    def value(xd, wd):
        z = xd @ wd.T
        lse = torch.logsumexp(z, 1)
        return ((lse - z.gather(1, targets[:, None])[:, 0]) * dloss.double() + lse * dlse.double()).sum()

    gen = torch.Generator().manual_seed(1)
    u, v = torch.randn(M, K, generator=gen).double().to(DEV), torch.randn(V, K, generator=gen).double().to(DEV)
    for direction, got in (((u, 0 * v), (dx.double() * u).sum()), ((0 * u, v), (dw.double() * v).sum())):
        h = 1e-4
        slope = (value(x.double() + h * direction[0], head.double() + h * direction[1])
                 - value(x.double() - h * direction[0], head.double() - h * direction[1])) / (2 * h)
        size = (dx.double().abs() * direction[0].abs()).sum() + (dw.double().abs() * direction[1].abs()).sum()
        assert (got - slope).abs() <= 2.0 ** -6 * size


def test_captured_and_replayed_beside_another_stream():
    M, V, K = 130, 3001, 264
    a, b = problem(M, V, K, 30), problem(M, V, K, 31)

    def step(x, head, targets, dloss, dlse):
        r = g.cross_entropy(x, head, targets)
        dx, dw = g.cross_entropy_backward(x, head, targets, r.lse, dloss, dlse=dlse, workspace=2 * M * 1024)
        return r.loss, r.lse, dx, dw

    want_a, want_b = step(*a), step(*b)
    static = [t.clone() for t in b]
    graphs = []
    for _ in range(2):  # two graphs of the same call: their workspaces are their own
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(*static)
        graphs.append((graph, out))
    for t, v in zip(static, a):
        t.copy_(v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
            got_b = step(*b)
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(u, v) for u, v in zip(out, want_a))
    assert all(torch.equal(u, v) for u, v in zip(got_b, want_b))


@pytest.mark.parametrize("M,V,K", [(1, 300, 64), (3, 5000, 520), (16, 1000, 264), (17, 2049, 72), (64, 4100, 1032)])
@pytest.mark.parametrize("workspace", [0, 1])
def test_few_rows_do_not_see_the_rounding_of_g(M, V, K, workspace):
    """Up to 64 rows G is the sum of two BF16 numbers: off by 2^-16 of itself instead of 2^-8."""
    x, head, targets, dloss, dlse = problem(M, V, K, M + K)
    wide = torch.zeros(M, K + 24, dtype=BF16, device=DEV)
    wide[:, 8:K + 8] = x
    x = wide[:, 8:K + 8]
    r = g.cross_entropy(x, head, targets)
    dx, dw = g.cross_entropy_backward(x, head, targets, r.lse, dloss, dlse=dlse, workspace=workspace)
    d = Definition(x, head, targets, 1.0)
    dl = dloss.double() * d.given
    a = (dl + dlse.double())[:, None] * (d.z - d.lse[:, None]).exp()
    G = a - dl[:, None] * d.onehot
    e = (d.E + d.lse.abs() * 2.0 ** -23 + 2.0 ** -19)[:, None]
    dG = e * a.abs() + 2.0 ** -16 * (G.abs() + e * a.abs())
    pieces = -(-V // g.cross_entropy_piece(M, V, workspace))
    for got, A, dA, B in ((dx, G, dG, d.w), (dw, G.T, dG.T, d.x)):
        want, size = A @ B, A.abs() @ B.abs()
        tol = dA @ B.abs() + (2 * A.shape[1] / 16 + 10 + 32 * pieces) * 2.0 ** -22 * size
        assert torch.all((got.double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol) + 1e-37)


@pytest.mark.parametrize("M", [40, 130, 700])
def test_gradient_takes_the_logits_that_the_forward_pass_took(M):
    """A target whose logit is one product of 2^24 and 480 steps of 16 products that add 1/2 each, a quarter of that number's
    last place: one accumulator never sees them, parts of the depth add them exactly. Every logit, its scale by 2^-20 and
    their difference to lse are exact then, so p is off by lse's rounding (half of 2^-19), the exponential's 2^-22 and its
    argument's product, less than 2^-20 + 2^-21 together; 1 - p is 3.4e-4."""
    K, V, scale = 8192, 3001, 2.0 ** -20
    x, head = torch.zeros(M, K), torch.zeros(V, K)
    x[:, 0], x[:, 512:] = 2.0 ** 12, 2.0 ** -5
    head[7, 0], head[7, 1:] = 2.0 ** 12, 1.0
    x, head = x.to(BF16).to(DEV), head.to(BF16).to(DEV)
    targets = torch.full((M,), 7, device=DEV)
    r = g.cross_entropy(x, head, targets, scale=scale)
    d = Definition(x, head, targets, scale)
    assert d.z[0, 7].item() == 16 + 240 * scale
    assert torch.all((r.lse.double() - d.lse).abs() <= 2.0 ** -20 + 2.0 ** -22)
    dx, dw = g.cross_entropy_backward(x, head, targets, r.lse, torch.full((M,), 1 / scale, device=DEV), scale=scale)
    p = (d.z - d.lse[:, None]).exp()
    G, e = p - d.onehot, (2.0 ** -20 + 2.0 ** -21) * p
    for got, A, dA, B in ((dx, G, e, d.w), (dw, G.T, e.T, d.x)):
        want, tol = A @ B, (dA + 2.0 ** -8 * (A.abs() + dA)) @ B.abs()
        assert torch.all((got.double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol) + 1e-37)


@pytest.mark.parametrize("M", [40, 200])
def test_long_sums_keep_their_digits(M):
    """Rows that lean on one target: its logit grows evenly over 4096 products. A tensor-core step cuts what is below its
    accumulator's last place, in the mean half of it, 2^-25 to 2^-24 of the accumulator; over n steps of an evenly growing sum
    that is n / 2 of these on one side. One accumulator (256 steps) would shrink the logit, and lse with it, by at least 3.8e-6;
    parts of 512 (32 steps) by 9.5e-7 at most, of 128 (8 steps, up to 64 rows) by 2.4e-7, and lse's rounding, 2^-24 on either
    side, is left with at most 2^-24 / sqrt(40) x 4 = 4e-8 of it in the mean.
    The target's share of G, p - 1 (read off a column of W that has a one in the target's row), is between 1/45 and 1/400 here,
    and z / (1 - p) 1420 and 2930 in the mean: in parts the logit's error and lse's move it by at most 9.5e-7 x 1420 = 1.4e-3
    of itself in the mean (up to 64 rows 2.4e-7 x 2930 = 7e-4), one accumulator by 5.4e-3 at least; G's and dX's roundings
    (2^-8 at most each, 1.7e-3 in the square mean) leave 4 x 2.4e-3 / sqrt(M) in the mean on top: 7e-4, at 40 rows 1.6e-3."""
    K, V, t = 4104, 2000, 7
    gen = torch.Generator().manual_seed(M)
    head = torch.randn(V, K, generator=gen) * 2 / K ** 0.5
    head[:, 4096:] = 0.0
    head[t, 4096] = 1.0
    x = torch.randn(M, K, generator=gen) * 0.02
    x += (2.9 + 0.4 * torch.rand(M, 1, generator=gen)) * head[t]
    x[:, 4096:] = 0.0
    x, head = x.to(BF16).to(DEV), head.to(BF16).to(DEV)
    targets = torch.full((M,), t, device=DEV)
    r = g.cross_entropy(x, head, targets)
    d = Definition(x, head, targets, 1.0)
    few = M <= 64
    assert ((r.lse.double() - d.lse) / d.lse).mean().abs() <= (3e-7 if few else 1e-6)
    dx, _ = g.cross_entropy_backward(x, head, targets, r.lse, torch.ones(M, device=DEV), weight_grad=False)
    share = (d.z[:, t] - d.lse).exp() - 1
    assert (d.z[:, t] / -share).mean() < (2930 if few else 1420)
    assert (dx[:, 4096].double() / share - 1).mean().abs() <= (2.4e-3 if few else 3.4e-3)


# where the gradient's products run on the 512 x 256 pair tile: in one piece with X copied to rows on 128-byte boundaries, in
# two pieces (the last one ragged) with such a copy, and in two without, of which the last one takes the 256 x 256 tile
LARGE = [(3500, 7501, 2056, 0, True, 512), (3500, 7001, 2056, 3584, True, 512), (2304, 4090, 2048, 2048, False, 256)]


@pytest.mark.parametrize("M,V,K,columns,copy,last", LARGE)
def test_the_large_tile(M, V, K, columns, copy, last):
    workspace = 2 * M * columns
    piece = g.cross_entropy_piece(M, V, workspace)
    for wave in range(68, 77):  # (whatever pairs the device holds)
        assert g.cross_entropy_plan(M, V, K, workspace, wave=wave) == (512, copy)
        assert g.cross_entropy_plan(M, (V - 1) % piece + 1, K, wave=wave)[0] == last
        if K == 2056:
            assert g.cross_entropy_plan(M, V, K, workspace, weight_grad=False, wave=wave)[0] == 512
            assert g.cross_entropy_plan(M, V, K, workspace, input_grad=False, wave=wave)[0] == 512
    x, head, targets, dloss, dlse = problem(M, V, K, M)
    r = g.cross_entropy(x, head, targets)
    d = Definition(x, head, targets, 1.0)
    d.check_forward(r)
    kw = dict(dlse=dlse, workspace=workspace)
    pieces = -(-V // piece)
    dx, dw = g.cross_entropy_backward(x, head, targets, r.lse, dloss, **kw)
    d.check_backward(dloss, dlse, dx, dw, pieces=pieces)
    again = g.cross_entropy_backward(x, head, targets, r.lse, dloss, **kw)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
    d.check_backward(dloss, dlse, *g.cross_entropy_backward(x, head, targets, r.lse, dloss, weight_grad=False, **kw),
                     pieces=pieces)
    d.check_backward(dloss, dlse, *g.cross_entropy_backward(x, head, targets, r.lse, dloss, input_grad=False, **kw),
                     pieces=pieces)
    assert g.get_device_status()[0] == 0


def test_a_copied_x_with_a_stride_and_what_lies_behind():
    M, V, K = 2500, 10500, 2008
    assert g.cross_entropy_plan(M, V, K)[1]
    x, head, targets, dloss, dlse = problem(M, V, K, 3)
    wide = torch.full((M + 1, K + 16), float("nan"), dtype=BF16, device=DEV)
    wide[:M, 8:K + 8] = x
    view = wide[:M, 8:K + 8]
    r, s = g.cross_entropy(x, head, targets), g.cross_entropy(view, head, targets)
    assert torch.equal(r.loss, s.loss) and torch.equal(r.lse, s.lse)
    want = g.cross_entropy_backward(x, head, targets, r.lse, dloss, dlse=dlse)
    got = g.cross_entropy_backward(view, head, targets, r.lse, dloss, dlse=dlse)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    Definition(x, head, targets, 1.0).check_backward(dloss, dlse, *got)


@pytest.mark.parametrize("M,V", [(70, 300), (600, 5003)])
def test_targets_outside_the_vocabulary_and_rows_of_nan_above_64_rows(M, V):
    x, head, targets, dloss, _ = problem(M, V, 64, 3)
    targets = targets.clamp(min=0)
    targets[1], targets[2], targets[M - 1] = V, -1, 1 << 40
    x[2], x[5, 3], x[M - 2, 63] = float("nan"), float("inf"), -float("inf")
    head[:, 63] = head[:, 63].abs() + 1  # (every logit of a row minus infinity)
    targets[5] = -1
    r = g.cross_entropy(x, head, targets)
    past = torch.zeros(M, dtype=torch.bool, device=DEV)
    past[[1, M - 1]] = True
    bad = torch.zeros_like(past)
    bad[[2, 5, M - 2]] = True
    assert torch.equal(r.lse.isnan(), bad)
    assert torch.equal(r.loss.isnan(), past | (bad & (targets >= 0))) and r.loss[2] == 0 and r.loss[5] == 0
    dx, _ = g.cross_entropy_backward(x, head, targets, r.lse, dloss, weight_grad=False)
    assert torch.equal(dx.isnan().any(1), past | (bad & (targets >= 0))) and torch.all(dx[[2, 5]] == 0)
