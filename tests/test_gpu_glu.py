"""gemm_glu_bf16, gemm_glu_e4m3 and the gradient through the binding, against FP64 evaluations of their definitions.

Tolerances, derived before the first run. FP32 accumulation of K products: at most K / 16 + 16 roundings or
truncations of partial sums no larger than S = sum |x w|, so the error of g (and u) is below
acc = (K / 16 + 16) 2^-23 S. H is rounded once (half a BF16 ulp, 2^-8 relative) from act(g) u, whose error is
|u| |act'| acc_g + |act| acc_u (|act'| < 1.2) plus the activation's own 2^-19. The gradients' products take dg
and du rounded to BF16: independent errors of at most 2^-8 of each term t, so their sum is within 8 standard
deviations, 8 / sqrt(3) 2^-8 sqrt(sum t^2), of the exact one; then one more rounding. Small integers make every
step exact and are compared bit for bit.
"""
import math

import pytest
import torch

import dense_tensor_core_persistent_gb300 as g
from dense_tensor_core_persistent_gb300 import build as gbuild

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
ACTS = ["silu", "gelu_tanh", "relu"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gbuild.build()


@pytest.fixture(autouse=True)
def _status():
    yield
    assert g.get_device_status() == (0, 0)


def act_fp64(x, act):
    if act == "silu":
        s = torch.sigmoid(x)
        return x * s, s * (1 + x * (1 - s))
    if act == "relu":
        return x.clamp(min=0), (x > 0).double()
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (x + 0.044715 * x ** 3))
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)


def problem(M, N, K, seed, std=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(M, K, generator=gen, device=DEV).to(torch.bfloat16)
    wg, wu = ((torch.randn(N, K, generator=gen, device=DEV) * std / math.sqrt(K)).to(torch.bfloat16) for _ in range(2))
    dh = torch.randn(M, N, generator=gen, device=DEV).to(torch.bfloat16)
    return x, wg, wu, dh


def check_forward(h, x, wg, wu, act):
    """x, wg, wu: FP64 values of the operands."""
    K = x.shape[1]
    gd, ud = x @ wg.T, x @ wu.T
    a, _ = act_fp64(gd, act)
    steps = (K / 16 + 16) * 2.0 ** -23
    acc_g, acc_u = steps * (x.abs() @ wg.abs().T), steps * (x.abs() @ wu.abs().T)
    want = a * ud
    tol = 2.0 ** -8 * want.abs() + 1.2 * ud.abs() * acc_g + a.abs() * acc_u + 2.0 ** -19 * want.abs() + 1e-30
    assert torch.all((h.double() - want).abs() <= tol * 1.01)
    return gd, ud


SHAPES = [(1, 8, 8), (1, 128, 64), (3, 264, 520), (5, 1000, 72), (16, 640, 1096), (17, 136, 4096), (33, 1368, 264),
          (64, 1024, 2048), (100, 72, 136), (128, 8, 8192), (129, 264, 128), (257, 136, 1032), (300, 1368, 520),
          (600, 2056, 256), (1030, 520, 392)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_forward(M, N, K, act):
    x, wg, wu, _ = problem(M, N, K, M + N + K)
    h = g.glu_bf16(x, wg, wu, act=act)
    gd, ud = check_forward(h, x.double(), wg.double(), wu.double(), act)
    h2, saved = g.glu_bf16(x, wg, wu, act=act, save=True)
    check_forward(h2, x.double(), wg.double(), wu.double(), act)
    steps = (K / 16 + 16) * 2.0 ** -23
    assert torch.all((saved[:, :N].double() - gd).abs() <= steps * (x.double().abs() @ wg.double().abs().T))
    assert torch.all((saved[:, N:].double() - ud).abs() <= steps * (x.double().abs() @ wu.double().abs().T))


@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (1, 136, 64), (2, 256, 4096), (4, 264, 528), (15, 72, 1040), (64, 1024, 2048), (20, 136, 784), (100, 72, 16),
                                   (130, 640, 272), (300, 1368, 528), (600, 520, 256)])
@pytest.mark.parametrize("act", ACTS)
def test_forward_e4m3(M, N, K, act):
    gen = torch.Generator(device=DEV).manual_seed(M * N + K)

    def rows(r, std):
        w = torch.randn(r, K, generator=gen, device=DEV) * std
        s = w.abs().amax(1) / 448
        return (w / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), s

    (x, xs), (wg, gs), (wu, us) = rows(M, 1.0), rows(N, 1 / math.sqrt(K)), rows(N, 1 / math.sqrt(K))
    h = g.glu_e4m3(x, xs, wg, gs, wu, us, act=act)
    check_forward(h, x.double() * xs.double()[:, None], wg.double() * gs.double()[:, None],
                  wu.double() * us.double()[:, None], act)


def gradient(dh, x, wg, wu, act):
    """FP64: dx, dwg, dwu and the root sums of squares of the terms of each."""
    x, wg, wu, dh = (t.double() for t in (x, wg, wu, dh))
    gd, ud = x @ wg.T, x @ wu.T
    a, da = act_fp64(gd, act)
    dg, du = dh * ud * da, dh * a
    grads = (dg @ wg + du @ wu, dg.T @ x, du.T @ x)
    sq = ((dg ** 2) @ (wg ** 2) + (du ** 2) @ (wu ** 2), (dg ** 2).T @ x ** 2, (du ** 2).T @ x ** 2)
    return grads, [s.sqrt() for s in sq]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_backward(M, N, K, act):
    x, wg, wu, dh = problem(M, N, K, 3 * M + N + K)
    _, saved = g.glu_bf16(x, wg, wu, act=act, save=True)
    got = g.glu_bf16_backward(dh, x, wg, wu, saved, act=act)
    if act == "relu":  # act' jumps at 0: take the kept g's side of it
        near = saved[:, :N].abs() < 1e-4
        dh = torch.where(near, 0.0, dh.float()).to(torch.bfloat16)
        got = g.glu_bf16_backward(dh, x, wg, wu, saved, act=act)
    want, root = gradient(dh, x, wg, wu, act)
    for a, b, r in zip(got, want, root):
        tol = 2.0 ** -8 * b.abs() + (8 / math.sqrt(3) * 2.0 ** -8 + 2.0 ** -10) * r + 1e-30
        assert a.shape == b.shape
        assert torch.all((a.double() - b).abs() <= tol)


def test_formula_against_differences():
    """The FP64 gradient above is that of sum(dH * H), by central differences."""
    M, N, K = 2, 8, 8
    x, wg, wu, dh = (t.double().cpu() for t in problem(M, N, K, 5))
    for act in ACTS:
        (dx, dwg, dwu), _ = gradient(dh, x, wg, wu, act)

        def value(x, wg, wu):
            return (dh * act_fp64(x @ wg.T, act)[0] * (x @ wu.T)).sum().item()

        h = 1e-6
        for t, grad, at in ((x, dx, 0), (wg, dwg, 1), (wu, dwu, 2)):
            for i in range(t.shape[0]):
                for j in range(t.shape[1]):
                    e = torch.zeros_like(t)
                    e[i, j] = h
                    plus = [x, wg, wu]
                    minus = [x, wg, wu]
                    plus[at], minus[at] = t + e, t - e
                    diff = (value(*plus) - value(*minus)) / (2 * h)
                    assert abs(diff - grad[i, j].item()) <= 1e-6 * (1 + abs(diff))


@pytest.mark.parametrize("M,N,K", [(300, 136, 64), (17, 264, 40), (515, 328, 64)])
def test_integers_bit_for_bit(M, N, K):
    """ReLU on small integers: g, u, dg, du are BF16 numbers and all sums are exact in FP32."""
    gen = torch.Generator(device=DEV).manual_seed(N)
    x = torch.randint(-2, 3, (M, K), generator=gen, device=DEV).to(torch.bfloat16)
    wg = torch.randint(-2, 3, (N, K), generator=gen, device=DEV).to(torch.bfloat16)
    wu = torch.randint(-2, 3, (N, K), generator=gen, device=DEV).to(torch.bfloat16)
    dh = torch.randint(-1, 2, (M, N), generator=gen, device=DEV).to(torch.bfloat16)
    h, saved = g.glu_bf16(x, wg, wu, act="relu", save=True)
    got = g.glu_bf16_backward(dh, x, wg, wu, saved, act="relu")
    gd, ud = x.double() @ wg.double().T, x.double() @ wu.double().T
    assert torch.equal(saved.double(), torch.cat((gd, ud), 1))
    assert torch.equal(h, (gd.clamp(min=0) * ud).to(torch.bfloat16))
    assert torch.equal(g.glu_bf16(x, wg, wu, act="relu"), h)
    want, _ = gradient(dh, x, wg, wu, "relu")
    for a, b in zip(got, want):
        assert torch.equal(a, b.to(torch.bfloat16))
    only = g.glu_bf16_backward(dh, x, wg, wu, saved, act="relu", weight_grads=False)
    assert only[1] is None and torch.equal(only[0], got[0])
    only = g.glu_bf16_backward(dh, x, wg, wu, saved, act="relu", input_grad=False)
    assert only[0] is None and torch.equal(only[1], got[1]) and torch.equal(only[2], got[2])


def test_strides():
    M, N, K = 37, 264, 136
    x, wg, wu, dh = problem(M, N, K, 71)
    wide = torch.full((M, K + 24), 7.0, dtype=torch.bfloat16, device=DEV)
    view = wide[:, 8:8 + K]
    view.copy_(x)
    dwide = torch.full((M, N + 16), 7.0, dtype=torch.bfloat16, device=DEV)
    dview = dwide[:, :N]
    dview.copy_(dh)
    h, saved = g.glu_bf16(x, wg, wu, save=True)
    assert torch.equal(g.glu_bf16(view, wg, wu), h)
    want = g.glu_bf16_backward(dh, x, wg, wu, saved)
    got = g.glu_bf16_backward(dview, view, wg, wu, saved)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = torch.full((M, N + 8), 3.0, dtype=torch.bfloat16, device=DEV)
    dx = torch.full((M, K + 8), 3.0, dtype=torch.bfloat16, device=DEV)
    g.gemm_glu_bf16(x, wg, wu, out, None, M, N, K, strides=g.gemm_glu_strides_t(0, N + 8, 0, 0))
    g.gemm_glu_bf16_backward(dh, x, wg, wu, saved, dx, None, None, M, N, K, strides=g.gemm_glu_strides_t(0, 0, 0, K + 8))
    assert torch.equal(out[:, :N], h) and torch.all(out[:, N:] == 3.0)
    assert torch.equal(dx[:, :K], want[0]) and torch.all(dx[:, K:] == 3.0)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [3, 200])
def test_extreme_values(act, M):
    """Large pre-activations saturate without NaN; a NaN row stays in its row."""
    N, K = 64, 64
    x, wg, wu, dh = problem(M, N, K, 13, std=300.0)
    h, saved = g.glu_bf16(x, wg, wu, act=act, save=True)
    assert torch.isfinite(h.float()).all()
    got = g.glu_bf16_backward(dh, x, wg, wu, saved, act=act)
    assert all(torch.isfinite(t.float()).all() for t in got)
    big = x.clone()
    big[1] = 1e30
    h = g.glu_bf16(big, wg.abs(), wu.abs(), act=act)
    assert torch.all(h[1] == math.inf) and torch.isfinite(h[[0, 2]].float()).all()
    bad = x.clone()
    bad[1, 3] = math.nan
    h2, s2 = g.glu_bf16(bad, wg, wu, act=act, save=True)
    assert h2[1].isnan().all() and torch.equal(h2[[0, 2]], g.glu_bf16(x, wg, wu, act=act)[[0, 2]])
    dx = g.glu_bf16_backward(dh, bad, wg, wu, s2, act=act, weight_grads=False)[0]
    assert dx[1].isnan().all() and torch.isfinite(dx[[0, 2]].float()).all()


def test_empty_sizes_stream_and_graph():
    x, wg, wu, dh = problem(40, 264, 136, 91)
    h, saved = g.glu_bf16(x, wg, wu, save=True)
    want = g.glu_bf16_backward(dh, x, wg, wu, saved)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    h2, s2 = g.glu_bf16(x, wg, wu, save=True, stream=side)
    got = g.glu_bf16_backward(dh, x, wg, wu, s2, stream=side)
    side.synchronize()
    assert torch.equal(h, h2) and all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h3, s3 = g.glu_bf16(x, wg, wu, save=True)
        got = g.glu_bf16_backward(dh, x, wg, wu, s3)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, h3) and all(torch.equal(a, b) for a, b in zip(got, want))
    e = torch.empty(0, 136, dtype=torch.bfloat16, device=DEV)
    he, se = g.glu_bf16(e, wg, wu, save=True)
    dx, dwg, dwu = g.glu_bf16_backward(he, e, wg, wu, se)
    assert he.shape == (0, 264) and dx.shape == (0, 136) and torch.all(dwg == 0) and torch.all(dwu == 0)
    z = torch.empty(5, 0, dtype=torch.bfloat16, device=DEV)
    w0 = torch.empty(264, 0, dtype=torch.bfloat16, device=DEV)
    assert torch.all(g.glu_bf16(z, w0, w0) == 0)
    n0 = torch.empty(0, 136, dtype=torch.bfloat16, device=DEV)
    dx = torch.ones(40, 136, dtype=torch.bfloat16, device=DEV)
    g.gemm_glu_bf16_backward(None, x, n0, n0, None, dx, None, None, 40, 0, 136)
    assert torch.all(dx == 0)


def test_many_tiles_per_cluster_repeat_bit_for_bit():
    """More tiles than co-resident pairs, several per pair, twice."""
    M, N, K = 2100, 7000, 520
    x, wg, wu, dh = problem(M, N, K, 17)
    h, saved = g.glu_bf16(x, wg, wu, save=True)
    check_forward(h, x.double(), wg.double(), wu.double(), "silu")
    got = g.glu_bf16_backward(dh, x, wg, wu, saved)
    again = g.glu_bf16_backward(dh, x, wg, wu, saved)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    want, root = gradient(dh, x, wg, wu, "silu")
    for a, b, r in zip(got, want, root):
        assert torch.all((a.double() - b).abs() <= 2.0 ** -8 * b.abs() + (8 / math.sqrt(3) * 2.0 ** -8 + 2.0 ** -10) * r)


@pytest.mark.parametrize("M,N,K,act", [(2500, 7000, 2056, "silu"), (3000, 2600, 4104, "gelu_tanh"),
                                       (3077, 5128, 2312, "silu")])
def test_large_tiles(M, N, K, act):
    """Ragged problems on the 512 x 256 pair tile, forward and backward, each against FP64 and twice bit for bit."""
    assert g.glu_plan(M, N, K) == (512, 512)
    x, wg, wu, dh = problem(M, N, K, M + K)
    check_forward(g.glu_bf16(x, wg, wu, act=act), x.double(), wg.double(), wu.double(), act)
    h, saved = g.glu_bf16(x, wg, wu, act=act, save=True)
    gd, ud = check_forward(h, x.double(), wg.double(), wu.double(), act)
    steps = (K / 16 + 16) * 2.0 ** -23
    assert torch.all((saved[:, :N].double() - gd).abs() <= steps * (x.double().abs() @ wg.double().abs().T))
    assert torch.all((saved[:, N:].double() - ud).abs() <= steps * (x.double().abs() @ wu.double().abs().T))
    got = g.glu_bf16_backward(dh, x, wg, wu, saved, act=act)
    want, root = gradient(dh, x, wg, wu, act)
    for a, b, r in zip(got, want, root):
        assert torch.all((a.double() - b).abs() <= 2.0 ** -8 * b.abs() + (8 / math.sqrt(3) * 2.0 ** -8 + 2.0 ** -10) * r)
    again = g.glu_bf16_backward(dh, x, wg, wu, saved, act=act)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    only = g.glu_bf16_backward(dh, x, wg, wu, saved, act=act, weight_grads=False)[0]
    assert torch.all((only.double() - want[0]).abs() <= 2.0 ** -8 * want[0].abs() + 0.02 * root[0])
    only = g.glu_bf16_backward(dh, x, wg, wu, saved, act=act, input_grad=False)[1:]
    for a, b, r in zip(only, want[1:], root[1:]):
        assert torch.all((a.double() - b).abs() <= 2.0 ** -8 * b.abs() + 0.02 * r)


@pytest.mark.parametrize("M,N,K", [(1, 512, 4096), (64, 64, 8192), (17, 1024, 1096), (100, 1792, 2056), (128, 4096, 520),
                                   (2, 2304, 1288), (33, 2432, 640)])
def test_few_rows_with_the_depth_shared(M, N, K):
    """Weights with few features: up to 8 CTAs share a tile's depth (here also in uneven parts)."""
    x, wg, wu, _ = problem(M, N, K, 7 * M + N + K)
    xd, gd, ud = x.double(), wg.double(), wu.double()
    h, saved = g.glu_bf16(x, wg, wu, save=True)
    gate, up = check_forward(h, xd, gd, ud, "silu")
    steps = (K / 16 + 16) * 2.0 ** -23
    assert torch.all((saved[:, :N].double() - gate).abs() <= steps * (xd.abs() @ gd.abs().T))
    assert torch.all((saved[:, N:].double() - up).abs() <= steps * (xd.abs() @ ud.abs().T))
    assert torch.equal(h, g.glu_bf16(x, wg, wu))  # the same bits again

    def rows(t):
        s = t.float().abs().amax(1) / 448
        return (t.float() / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), s

    if K % 16 == 0:
        (xe, xs), (ge, gs), (ue, us) = rows(x), rows(wg), rows(wu)
        h = g.glu_e4m3(xe, xs, ge, gs, ue, us)
        check_forward(h, xe.double() * xs.double()[:, None], ge.double() * gs.double()[:, None],
                      ue.double() * us.double()[:, None], "silu")


def test_few_rows_with_the_depth_shared_exact():
    """Small integers: every partial sum is exact, and so is the join."""
    gen = torch.Generator(device=DEV).manual_seed(3)
    x, wg, wu = (torch.randint(-2, 3, s, generator=gen, device=DEV).to(torch.bfloat16)
                 for s in ((40, 1544), (1000, 1544), (1000, 1544)))
    _, saved = g.glu_bf16(x, wg, wu, act="relu", save=True)
    assert torch.equal(saved[:, :1000].double(), x.double() @ wg.double().T)
    assert torch.equal(saved[:, 1000:].double(), x.double() @ wu.double().T)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 264), (6, 2648, 824), (33, 4096, 136), (257, 2056, 520), (512, 4096, 1024)])
def test_backward_with_dx_in_slices(M, N, K):
    """Few tiles of dX and a long sum: partial sums of slices, with dX alone and beside dW, the same bits again."""
    x, wg, wu, dh = problem(M, N, K, 5 * M + N + K)
    _, saved = g.glu_bf16(x, wg, wu, save=True)
    got = g.glu_bf16_backward(dh, x, wg, wu, saved)
    want, root = gradient(dh, x, wg, wu, "silu")
    for a, b, r in zip(got, want, root):
        tol = 2.0 ** -8 * b.abs() + (8 / math.sqrt(3) * 2.0 ** -8 + 2.0 ** -10) * r + 1e-30
        assert torch.all((a.double() - b).abs() <= tol)
    again = g.glu_bf16_backward(dh, x, wg, wu, saved)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    alone, _, _ = g.glu_bf16_backward(dh, x, wg, wu, saved, weight_grads=False)
    tol = 2.0 ** -8 * want[0].abs() + (8 / math.sqrt(3) * 2.0 ** -8 + 2.0 ** -10) * root[0] + 1e-30
    assert torch.all((alone.double() - want[0]).abs() <= tol)


def e4m3_rows(t):
    s = t.float().abs().amax(1) / 448
    return (t.float() / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), s


def check_e4m3(x, wg, wu, act="silu"):
    """The E4M3 form on the quantised operands, against FP64."""
    (xe, xs), (ge, gs), (ue, us) = e4m3_rows(x), e4m3_rows(wg), e4m3_rows(wu)
    h = g.glu_e4m3(xe, xs, ge, gs, ue, us, act=act)
    check_forward(h, xe.double() * xs.double()[:, None], ge.double() * gs.double()[:, None],
                  ue.double() * us.double()[:, None], act)


@pytest.mark.parametrize("M,N,K", [(1, 20016, 144), (20, 19464, 272), (64, 29192, 80), (100, 20008, 144), (128, 19520, 208),
                                   (33, 16128, 1040)])
def test_few_rows_with_several_tiles_a_cta(M, N, K):
    """More tiles of 64 features than SMs: second and later items of a CTA, with halves in the last wave and (16128)
    without."""
    x, wg, wu, _ = problem(M, N, K, M + N + K)
    xd, gd, ud = x.double(), wg.double(), wu.double()
    h, saved = g.glu_bf16(x, wg, wu, act="gelu_tanh", save=True)
    gate, up = check_forward(h, xd, gd, ud, "gelu_tanh")
    steps = (K / 16 + 16) * 2.0 ** -23
    assert torch.all((saved[:, :N].double() - gate).abs() <= steps * (xd.abs() @ gd.abs().T))
    assert torch.all((saved[:, N:].double() - up).abs() <= steps * (xd.abs() @ ud.abs().T))
    assert torch.equal(h, g.glu_bf16(x, wg, wu, act="gelu_tanh"))
    check_e4m3(x, wg, wu, "gelu_tanh")


@pytest.mark.parametrize("M,N,K", [(300, 12800, 272), (300, 10880, 528), (1030, 5128, 272), (129, 19464, 144),
                                   (2000, 2568, 2064)])
@pytest.mark.parametrize("act", ["silu", "relu"])
def test_e4m3_with_several_tiles_a_pair(M, N, K, act):
    """Whole tiles of the pair tile in E4M3, and more of them than pairs (10880, 19464: a last wave of halves)."""
    x, wg, wu, _ = problem(M, N, K, M + N + K)
    check_e4m3(x, wg, wu, act)


@pytest.mark.parametrize("M,N,K", [(128, 264, 136), (300, 264, 136), (2500, 7000, 2056)])
def test_strides_on_each_tile(M, N, K):
    """X, H, dH and dX with rows apart from one another, on the few-row kernel, the pair tile and the 512 x 256 one."""
    assert g.glu_plan(M, N, K) == {128: (0, 256), 300: (256, 256), 2500: (512, 512)}[M]
    x, wg, wu, dh = problem(M, N, K, 73)
    h, saved = g.glu_bf16(x, wg, wu, save=True)
    want = g.glu_bf16_backward(dh, x, wg, wu, saved)

    def apart(t, before, after):
        wide = torch.full((M, before + t.shape[1] + after), 7.0, dtype=t.dtype, device=DEV)
        wide[:, before:before + t.shape[1]] = t
        return wide[:, before:before + t.shape[1]]

    xv, dhv = apart(x, 8, 16), apart(dh, 0, 40)
    h2, saved2 = g.glu_bf16(xv, wg, wu, save=True)
    assert torch.equal(h2, h) and torch.equal(saved2, saved)
    assert all(torch.equal(a, b) for a, b in zip(g.glu_bf16_backward(dhv, xv, wg, wu, saved), want))
    out, dx = (torch.full((M, n + 24), 3.0, dtype=torch.bfloat16, device=DEV) for n in (N, K))
    g.gemm_glu_bf16(x, wg, wu, out, None, M, N, K, strides=g.gemm_glu_strides_t(0, N + 24, 0, 0))
    g.gemm_glu_bf16_backward(dh, x, wg, wu, saved, dx, *(torch.empty_like(wg) for _ in range(2)), M, N, K,
                             strides=g.gemm_glu_strides_t(0, 0, 0, K + 24))
    assert torch.equal(out[:, :N], h) and torch.all(out[:, N:] == 3.0)
    assert torch.equal(dx[:, :K], want[0]) and torch.all(dx[:, K:] == 3.0)


@pytest.mark.parametrize("M", [37, 300])
def test_e4m3_strides(M):
    N, K = 264, 144
    x, wg, wu, _ = problem(M, N, K, 79)
    (xe, xs), (ge, gs), (ue, us) = e4m3_rows(x), e4m3_rows(wg), e4m3_rows(wu)
    want = g.glu_e4m3(xe, xs, ge, gs, ue, us)
    wide = torch.full((M, K + 48), 7.0, device=DEV).to(torch.float8_e4m3fn)
    view = wide[:, 16:16 + K]
    view.copy_(xe)
    assert torch.equal(g.glu_e4m3(view, xs, ge, gs, ue, us), want)
    out = torch.full((M, N + 16), 3.0, dtype=torch.bfloat16, device=DEV)
    g.gemm_glu_e4m3(view, xs, ge, gs, ue, us, out, M, N, K, strides=g.gemm_glu_strides_t(K + 48, N + 16, 0, 0))
    assert torch.equal(out[:, :N], want) and torch.all(out[:, N:] == 3.0)
