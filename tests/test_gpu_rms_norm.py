"""gemm_rms_norm and its gradient through the binding, against FP64 evaluations of their definitions.

Tolerances, derived before the first run. The stream s = bf16(x + r) is compared exactly. A BF16
output lies within half a BF16 ulp of the FP32 result, that is 2^-8 of its magnitude at most; the
FP32 evaluation before it (the sum of squares over up to 32760 terms added in a tree of depth < 48,
a square root, a division, three products) adds less than 2^-17 of the magnitude. The gradient's
terms cancel, so its FP32 error is bounded by the magnitudes of the terms it adds. An 8-bit or 4-bit
code is the rounding of a value that carries the FP32 error: the decoded value is the nearest one or,
within that error of a tie, its neighbour, so |decoded - y| is at most half the code's step plus the
FP32 error.
"""
import math

import pytest
import torch

import dense_tensor_core_persistent_gb300 as g
import oracle
import synthetic_inputs as si
from dense_tensor_core_persistent_gb300 import build as gbuild

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
FP32_REL = 2.0 ** -17
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gbuild.build()


def rand(seed, *shape, std=1.0):
    t = torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std
    return t.to(torch.bfloat16)


def problem(rows, cols, seed, residual=True):
    x = rand(seed, rows, cols)
    r = rand(seed + 1, rows, cols, std=3.0) if residual else None
    w = (1 + 0.3 * torch.randn(cols, generator=torch.Generator().manual_seed(seed + 2))).to(torch.bfloat16)
    return x, r, w


def definition(x, r, w, eps=EPS):
    s = x if r is None else (x.float() + r.float()).to(torch.bfloat16)
    sd = s.double()
    rstd = 1 / (sd.square().mean(1, keepdim=True) + eps).sqrt()
    y = sd * rstd
    return s, rstd, y if w is None else y * w.double()


def dev(t):
    return None if t is None else t.to(DEV)


SHAPES = [(1, 1), (1, 8192), (3, 7), (2, 8), (5, 15), (17, 4099), (700, 520), (2, 16391), (3, 32760), (1300, 64),
          (4, 16384), (2500, 1032), (33, 4104), (1, 9), (64, 2049)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_bf16(rows, cols, residual):
    x, r, w = problem(rows, cols, rows + cols, residual)
    n = g.rms_norm(dev(x), dev(w), residual=dev(r), eps=EPS, save=True)
    s, rstd, y = definition(x, r, w)
    assert torch.equal(n.sum.cpu(), s)
    assert torch.all((n.rstd.cpu().double() - rstd[:, 0]).abs() <= FP32_REL * rstd[:, 0])
    assert torch.all((n.y.cpu().double() - y).abs() <= (2.0 ** -8 + FP32_REL) * y.abs())


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_e4m3(rows, cols):
    x, r, w = problem(rows, cols, 3 * rows + cols)
    n = g.rms_norm(dev(x), dev(w), residual=dev(r), eps=EPS, out="e4m3")
    s, _, y = definition(x, r, w)
    assert torch.equal(n.sum.cpu(), s)
    scale = y.abs().amax(1) / 448
    got_scale = n.scales.cpu().double()
    assert torch.all((got_scale - scale).abs() <= FP32_REL * scale)
    q = y / got_scale[:, None]
    # half a step: 2^-4 of the binade's lowest value from 2^-6 up, 2^-10 below
    half = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 4)
    code = n.y.cpu().double()
    assert code.abs().max() <= 448
    assert torch.all((code - q).abs() <= half + 2 * FP32_REL * q.abs())


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 256), (129, 4096), (5, 32752), (1000, 512)])
def test_nvfp4(rows, cols):
    x, r, w = problem(rows, cols, rows + 7 * cols)
    n = g.rms_norm(dev(x), dev(w), residual=dev(r), eps=EPS, out="nvfp4")
    s, _, y = definition(x, r, w)
    assert torch.equal(n.sum.cpu(), s)
    blocks = y.view(rows, -1, 16)
    ideal = blocks.abs().amax(2) / 6
    sf = n.scales.cpu().view(torch.float8_e4m3fn).double()
    half = torch.exp2(torch.floor(torch.log2(ideal.clamp(min=2.0 ** -6))) - 4)
    assert torch.all((sf - ideal).abs() <= half + FP32_REL * ideal)
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
    b = n.y.cpu()
    code = torch.stack((table[(b & 15).long()], table[(b >> 4).long()]), 2).view(rows, -1, 16)
    q = (blocks / sf[:, :, None]).clamp(-6, 6)
    step = torch.where(q.abs() < 2, 0.5, torch.where(q.abs() < 4, 1.0, 2.0))
    assert torch.all((code - q).abs() <= step / 2 + 2 * FP32_REL * q.abs())


def test_nvfp4_feeds_the_product():
    """y and scales are A and SFA of matmul_nvfp4: the product of the decoded operands."""
    M, N, K = 70, 264, 512
    x, r, w = problem(M, K, 5)
    _, _, b, sfb = si.nvfp4_problem(9, M, N, K)
    n = g.rms_norm(dev(x), dev(w), residual=dev(r), out="nvfp4")
    C = g.matmul_nvfp4(n.y, n.scales, b.to(DEV), sfb.to(DEV))
    ref = torch.from_numpy(oracle.gemm_nvfp4(n.y.cpu(), n.scales.cpu(), b, sfb))
    # one BF16 rounding, and FP32 accumulation over 512 products
    assert torch.all((C.cpu().double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-5 * ref.abs().max())


@pytest.mark.parametrize("out", ["bf16", "e4m3"])
def test_strides_and_offsets(out):
    """Columns of a wider matrix, at offsets that share and that do not share their misalignment."""
    rows, cols = 37, 1003
    for off_x, off_r, wide in ((0, 0, 1008), (3, 3, 1011), (1, 6, 1010), (8, 0, 1024)):
        x, r, w = problem(rows, cols, 11 * off_x + off_r)
        bx, br = torch.full((rows, wide + 8), 9.0, dtype=torch.bfloat16, device=DEV), torch.full(
            (rows, wide + 8), 9.0, dtype=torch.bfloat16, device=DEV)
        vx, vr = bx[:, off_x:off_x + cols], br[:, off_r:off_r + cols]
        vx.copy_(x)
        vr.copy_(r)
        n = g.rms_norm(vx, dev(w), residual=vr, out=out, inplace=True)
        s, _, y = definition(x, r, w)
        assert n.sum.data_ptr() == vr.data_ptr()
        assert torch.equal(vr.cpu(), s)
        assert torch.equal(vx.cpu(), x)
        outside = torch.ones(wide + 8, dtype=torch.bool)
        outside[off_r:off_r + cols] = False
        assert torch.all(br[:, outside.to(DEV)] == 9.0)
        plain = g.rms_norm(dev(x), dev(w), residual=dev(r), out=out)
        if out == "bf16":
            assert torch.all((n.y.cpu().double() - y).abs() <= (2.0 ** -8 + FP32_REL) * y.abs())
        else:
            got, want = (t.y.cpu().double() * t.scales.cpu().double()[:, None] for t in (n, plain))
            assert torch.all((got - y).abs() <= y.abs() * 2.0 ** -4 + y.abs().amax(1, keepdim=True) * 2.0 ** -9 / 448)
            assert torch.all((want - y).abs() <= y.abs() * 2.0 ** -4 + y.abs().amax(1, keepdim=True) * 2.0 ** -9 / 448)


def test_rows_with_zeros_infinities_and_nan():
    rows, cols = 6, 264
    x, _, w = problem(rows, cols, 21, residual=False)
    x[1] = 0.0
    x[2, 5] = math.inf
    x[3, 7] = math.nan
    x[4] = 3.0e38  # the squares overflow FP32
    for c in (cols, 257):
        xs = x[:, :c].contiguous()
        got = g.rms_norm(dev(xs), dev(w[:c].contiguous())).y.cpu().float()
        f = xs.float()
        want = f * (1 / torch.sqrt((f * f).mean(1, keepdim=True) + EPS)) * w[:c].float()
        assert torch.equal(got.isnan(), want.isnan())
        fine = ~want.isnan()
        assert torch.all((got - want)[fine].abs() <= 2.0 ** -7 * want[fine].abs())
        assert torch.all(got[1] == 0)
        n = g.rms_norm(dev(xs), dev(w[:c].contiguous()), out="e4m3")
        sc = n.scales.cpu()
        assert sc[1] == 0 and torch.all(n.y[1].cpu().float() == 0)
        assert sc[2].isnan() and sc[3].isnan() and sc[0].isfinite() and sc[5].isfinite()
        assert not n.y.cpu().float()[[0, 1, 5]].isnan().any()


def backward_definition(dy, s, w, ds, eps=EPS):
    sd, d = s.double(), dy.double()
    rstd = 1 / (sd.square().mean(1, keepdim=True) + eps).sqrt()
    xh, dyw = sd * rstd, d * w.double()
    c = (dyw * xh).mean(1, keepdim=True)
    dx = rstd * (dyw - xh * c) + (0 if ds is None else ds.double())
    terms = rstd * (dyw.abs() + (xh * c).abs() + xh.abs() * (dyw * xh).abs().mean(1, keepdim=True))
    dw = (d * xh).sum(0)
    return dx, terms + (0 if ds is None else ds.double().abs()), dw, (d * xh).abs().sum(0)


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("past", [True, False])
def test_backward(rows, cols, past):
    x, r, w = problem(rows, cols, 5 * rows + cols)
    dy = rand(rows, rows, cols)
    ds = rand(cols + 1, rows, cols, std=0.5) if past else None
    n = g.rms_norm(dev(x), dev(w), residual=dev(r), eps=EPS, save=True)
    dx, dw = g.rms_norm_backward(dev(dy), n.sum, dev(w), n.rstd, dsum=dev(ds))
    want, terms, want_dw, terms_dw = backward_definition(dy, n.sum.cpu(), w, ds)
    assert torch.all((dx.cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + FP32_REL * terms)
    # rows are added within CTAs, then over at most 1216 CTAs in eight chains: fewer than 2^9 roundings deep here
    assert torch.all((dw.cpu().double() - want_dw).abs() <= 2.0 ** -14 * terms_dw + 1e-30)


def test_backward_against_differences():
    """The gradient of sum(dy * y) by central differences of the FP64 definition."""
    rows, cols = 2, 24
    x, _, w = problem(rows, cols, 77, residual=False)
    dy = rand(78, rows, cols)
    n = g.rms_norm(dev(x), dev(w), save=True)
    dx, dw = g.rms_norm_backward(dev(dy), n.sum, dev(w), n.rstd)

    def value(xd, wd):
        return (dy.double() * xd / (xd.square().mean(1, keepdim=True) + 1e-5).sqrt() * wd).sum()

    h = 1e-5
    for i in range(rows):
        for j in range(0, cols, 5):
            e = torch.zeros(rows, cols, dtype=torch.float64)
            e[i, j] = h
            diff = (value(x.double() + e, w.double()) - value(x.double() - e, w.double())) / (2 * h)
            assert abs(dx[i, j].item() - diff.item()) <= 2.0 ** -8 * abs(diff.item()) + 1e-5
    for j in range(cols):
        e = torch.zeros(cols, dtype=torch.float64)
        e[j] = h
        diff = (value(x.double(), w.double() + e) - value(x.double(), w.double() - e)) / (2 * h)
        assert abs(dw[j].item() - diff.item()) <= 1e-5 * (1 + abs(diff.item()))


def test_backward_repeats_bit_for_bit_and_in_place():
    rows, cols = 3001, 1027
    x, r, w = problem(rows, cols, 31)
    dy, ds = rand(32, rows, cols), rand(33, rows, cols)
    n = g.rms_norm(dev(x), dev(w), residual=dev(r), save=True)
    dx, dw = g.rms_norm_backward(dev(dy), n.sum, dev(w), n.rstd, dsum=dev(ds))
    dx2, dw2 = g.rms_norm_backward(dev(dy), n.sum, dev(w), n.rstd, dsum=dev(ds))
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    acc = dev(ds)
    g.gemm_rms_norm_backward(dev(dy), n.sum, dev(w), n.rstd, acc, acc, None, rows, cols)
    assert torch.equal(acc, dx)


def test_empty_and_other_stream():
    w = torch.ones(16, dtype=torch.bfloat16, device=DEV)
    n = g.rms_norm(torch.empty(0, 16, dtype=torch.bfloat16, device=DEV), w, save=True)
    assert n.y.shape == (0, 16)
    _, dw = g.rms_norm_backward(torch.empty(0, 16, dtype=torch.bfloat16, device=DEV), n.sum, w, n.rstd)
    assert torch.all(dw == 0)
    x, r, wt = problem(65, 776, 41)
    xd, rd, wd = dev(x), dev(r), dev(wt)
    want = g.rms_norm(xd, wd, residual=rd)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = g.rms_norm(xd, wd, residual=rd, stream=side)
    side.synchronize()
    assert torch.equal(got.y, want.y) and torch.equal(got.sum, want.sum)


def test_graph_capture():
    x, r, w = problem(40, 1040, 51)
    xd, rd, wd, dy = dev(x), dev(r), dev(w), dev(rand(52, 40, 1040))
    n = g.rms_norm(xd, wd, residual=rd, save=True)
    want = (n.y, *g.rms_norm_backward(dy, n.sum, wd, n.rstd))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m = g.rms_norm(xd, wd, residual=rd, save=True)
        got = (m.y, *g.rms_norm_backward(dy, m.sum, wd, m.rstd))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("cols", [520, 1003, 16391])
@pytest.mark.parametrize("weight", [2.0 ** -118, 2.0 ** -122, 2.0 ** -126, 2.0 ** -131])
def test_e4m3_of_tiny_rows(cols, weight):
    """Rows near FP32's smallest normal number: the scale stops at 2^-127, and codes and scale still belong together."""
    rows = 5
    x, _, w = problem(rows, cols, cols, residual=False)
    w = (w.float() * weight).to(torch.bfloat16)
    w[3] = 0.0
    n = g.rms_norm(dev(x), dev(w), eps=EPS, out="e4m3")
    _, _, y = definition(x, None, w)
    got = n.scales.cpu().double()
    tiny = 2.0 ** -149
    assert torch.all((got - (y.abs().amax(1) / 448).clamp(min=2.0 ** -127)).abs() <= FP32_REL * got + tiny)
    q = (y / got[:, None]).clamp(-448, 448)
    half = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 4)
    # y itself is a product of FP32 numbers, at its smallest in steps of 2^-149
    assert torch.all((n.y.cpu().double() - q).abs() <= half + 2 * FP32_REL * q.abs() + 2 * tiny / got[:, None])


def test_rows_without_columns():
    """Rows of no columns: nothing to norm, a scale and an rstd of 0."""
    x = torch.empty(300, 0, dtype=torch.bfloat16, device=DEV)
    scales, rstd = torch.full((300,), 7.0, device=DEV), torch.full((300,), 7.0, device=DEV)
    g.gemm_rms_norm(x, None, None, None, x, scales, rstd, 300, 0, EPS, g.GEMM_NORM_E4M3)
    assert torch.all(scales == 0) and torch.all(rstd == 0)
    rstd.fill_(7.0)
    g.gemm_rms_norm(x, None, None, None, x, None, rstd, 300, 0, EPS)
    assert torch.all(rstd == 0)
    n = g.rms_norm(x, save=True)
    assert n.y.shape == (300, 0)
    dx, dw = g.rms_norm_backward(x, n.sum, None, n.rstd)
    assert dx.shape == (300, 0) and dw.shape == (0,)


# Widths of two, four and eight groups a thread, on the 16-byte boundary and off it, with more rows than resident CTAs.
SEVERAL_ROWS = [(1500, 4096), (2000, 2051), (400, 12000), (400, 12003), (330, 20000), (330, 20001)]


@pytest.mark.parametrize("rows,cols", SEVERAL_ROWS)
def test_several_rows_a_cta(rows, cols):
    test_bf16(rows, cols, True)
    test_e4m3(rows, cols)
    test_backward(rows, cols, True)


@pytest.mark.parametrize("rows,cols", [(6000, 256), (1500, 4096), (400, 12000), (330, 20000)])
def test_nvfp4_with_several_rows_a_cta(rows, cols):
    test_nvfp4(rows, cols)


@pytest.mark.parametrize("cols", [1003, 9001])
def test_several_rows_a_cta_that_share_no_alignment(cols):
    """x, the residual and the gradients at offsets and strides of their own: element by element."""
    rows = 1300
    x, r, w = problem(rows, cols, cols)
    dy, ds = rand(cols + 5, rows, cols), rand(cols + 6, rows, cols, std=0.5)

    def apart(t, before, wide):
        v = torch.full((rows, wide), 9.0, dtype=torch.bfloat16, device=DEV)[:, before:before + cols]
        v.copy_(t)
        return v

    vx, vr = apart(x, 1, cols + 7), apart(r, 6, cols + 9)
    n = g.rms_norm(vx, dev(w), residual=vr, eps=EPS, save=True)
    s, rstd, y = definition(x, r, w)
    assert torch.equal(n.sum.cpu(), s)
    assert torch.all((n.rstd.cpu().double() - rstd[:, 0]).abs() <= FP32_REL * rstd[:, 0])
    assert torch.all((n.y.cpu().double() - y).abs() <= (2.0 ** -8 + FP32_REL) * y.abs())
    dx, dw = g.rms_norm_backward(apart(dy, 3, cols + 4), apart(s, 2, cols + 5), dev(w), n.rstd, dsum=apart(ds, 5, cols + 12))
    want, terms, want_dw, terms_dw = backward_definition(dy, s, w, ds)
    assert torch.all((dx.cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + FP32_REL * terms)
    assert torch.all((dw.cpu().double() - want_dw).abs() <= 2.0 ** -14 * terms_dw + 1e-30)
