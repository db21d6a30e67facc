"""gemm_layer_norm and its gradient through the binding, against FP64 evaluations of their definitions.

Tolerances, derived before the first run. The stream s = bf16(x + r) is compared exactly. The mean is an FP32 sum of up
to 32760 terms, fewer than 64 roundings deep: off by at most 2^-18 of the mean magnitude, e. The variance is a sum of
squared differences, each off by its rounding: 2^-17 of itself and, through the mean, e^2. So rstd is off by at most
R = 2^-17 + (e rstd)^2 + 2^-23 relative, and (s - mu) rstd by R of itself and e rstd. A BF16 output adds half a BF16 ulp, 2^-8
of its magnitude at most, and the affine step 2^-22 of its terms. The gradient's terms cancel, so its FP32 error is bounded
by the magnitudes of the terms it adds. An 8-bit or 4-bit code is the rounding of a value that carries the FP32 error: the
decoded value is off by at most half the code's step plus the FP32 error.
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
BF16 = torch.bfloat16
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gbuild.build()


def rand(seed, *shape, std=1.0):
    t = torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std
    return t.to(BF16)


def problem(rows, cols, seed, residual=True, mean=1.0):
    x = rand(seed, rows, cols)
    r = None
    if residual:
        at = mean * torch.randn(rows, 1, generator=torch.Generator().manual_seed(seed + 9))
        r = (rand(seed + 1, rows, cols, std=3.0).float() + at).to(BF16)
    w = (1 + 0.3 * torch.randn(cols, generator=torch.Generator().manual_seed(seed + 2))).to(BF16)
    return x, r, w, rand(seed + 3, cols, std=0.4)


class Definition:
    """y and what FP32 may cost it, from the rounded stream."""

    def __init__(self, x, r, w, b, eps=EPS):
        self.s = x if r is None else (x.float() + r.float()).to(BF16)
        sd = self.s.double()
        var, self.mean = torch.var_mean(sd, 1, correction=0, keepdim=True)
        self.rstd = 1 / (var + eps).sqrt()
        self.xh = (sd - self.mean) * self.rstd
        self.w = torch.ones(x.shape[1]).double() if w is None else w.double()
        self.b = torch.zeros(x.shape[1]).double() if b is None else b.double()
        self.y = self.xh * self.w + self.b
        self.e = 2.0 ** -18 * sd.abs().mean(1, keepdim=True)
        self.R = 2.0 ** -17 + (self.e * self.rstd) ** 2 + 2.0 ** -23
        self.e_xh = self.R * self.xh.abs() + self.e * self.rstd
        self.err = self.e_xh * self.w.abs() + 2.0 ** -22 * ((self.xh * self.w).abs() + self.b.abs())

    def check(self, n):
        assert torch.equal(n.sum.cpu(), self.s)
        if n.mean is not None:
            assert torch.all((n.mean.cpu().double()[:, None] - self.mean).abs() <= self.e)
            assert torch.all((n.rstd.cpu().double()[:, None] - self.rstd).abs() <= self.R * self.rstd)
        self.check_y(n.y)

    def check_y(self, y):
        assert torch.all((y.cpu().double() - self.y).abs() <= 2.0 ** -8 * self.y.abs() + 2 * self.err)

    def check_e4m3(self, n):
        assert torch.equal(n.sum.cpu(), self.s)
        scale, slack = self.y.abs().amax(1) / 448, self.err.amax(1) / 448
        got = n.scales.cpu().double()
        assert torch.all((got - scale).abs() <= 2.0 ** -22 * scale + slack)
        q = self.y / got[:, None]
        half = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 4)
        code = n.y.cpu().double()
        assert code.abs().max() <= 448
        assert torch.all((code - q).abs() <= half + 2 * self.err / got[:, None] + 2.0 ** -20 * q.abs())


def dev(t):
    return None if t is None else t.to(DEV)


SHAPES = [(1, 1), (1, 8192), (3, 7), (2, 8), (5, 15), (17, 4099), (700, 520), (2, 16391), (3, 32760), (1300, 64),
          (4, 16384), (2500, 1032), (33, 4104), (1, 9), (64, 2049)]
# two, four and eight groups a thread, on the 16-byte boundary and off it, with more rows than resident CTAs
SEVERAL_ROWS = [(1500, 4096), (2000, 2051), (1500, 8192), (400, 12000), (400, 12003), (330, 20000), (330, 20001),
                (200, 30719), (160, 30721), (3000, 16), (3000, 17), (5000, 257), (6000, 511), (5000, 23)]


@pytest.mark.parametrize("rows,cols", SHAPES + SEVERAL_ROWS)
@pytest.mark.parametrize("residual", [True, False])
def test_bf16(rows, cols, residual):
    x, r, w, b = problem(rows, cols, rows + cols, residual)
    Definition(x, r, w, b).check(g.layer_norm(dev(x), dev(w), dev(b), residual=dev(r), eps=EPS, save=True))


@pytest.mark.parametrize("rows,cols", [(5, 264), (3, 1001)])
def test_without_weight_or_bias(rows, cols):
    x, r, w, b = problem(rows, cols, cols)
    for wt, bt in ((None, None), (w, None), (None, b)):
        d = Definition(x, r, wt, bt)
        d.check(g.layer_norm(dev(x), dev(wt), dev(bt), residual=dev(r)))
        d.check_e4m3(g.layer_norm(dev(x), dev(wt), dev(bt), residual=dev(r), out="e4m3"))


@pytest.mark.parametrize("rows,cols", [(4, 520), (3, 1003), (200, 8192)])
@pytest.mark.parametrize("mean", [30.0, 3000.0])
def test_means_far_above_the_spread(rows, cols, mean):
    # the stream's own rounding leaves a few values next to the mean: their spread has to survive
    gen = torch.Generator().manual_seed(cols)
    x = (mean + 0.02 * mean * torch.randn(rows, cols, generator=gen)).to(BF16)
    _, _, w, b = problem(1, cols, 4)
    Definition(x, None, w, b).check(g.layer_norm(dev(x), dev(w), dev(b), save=True))
    same = torch.full((rows, cols), mean, dtype=BF16)
    n = g.layer_norm(dev(same), dev(w), dev(b), save=True)
    Definition(same, None, w, b).check(n)


@pytest.mark.parametrize("rows,cols", SHAPES + SEVERAL_ROWS)
def test_e4m3(rows, cols):
    x, r, w, b = problem(rows, cols, 3 * rows + cols)
    Definition(x, r, w, b).check_e4m3(g.layer_norm(dev(x), dev(w), dev(b), residual=dev(r), eps=EPS, out="e4m3"))


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 256), (129, 4096), (5, 32752), (6000, 256), (400, 12000)])
def test_nvfp4(rows, cols):
    x, r, w, b = problem(rows, cols, rows + 7 * cols)
    n = g.layer_norm(dev(x), dev(w), dev(b), residual=dev(r), eps=EPS, out="nvfp4")
    d = Definition(x, r, w, b)
    assert torch.equal(n.sum.cpu(), d.s)
    blocks, err = d.y.view(rows, -1, 16), d.err.view(rows, -1, 16)
    ideal, slack = blocks.abs().amax(2) / 6, err.amax(2) / 6
    sf = n.scales.cpu().view(torch.float8_e4m3fn).double()
    half = torch.exp2(torch.floor(torch.log2(ideal.clamp(min=2.0 ** -6))) - 4)
    assert torch.all((sf - ideal).abs() <= half + 2.0 ** -20 * ideal + 2 * slack)
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
    c = n.y.cpu()
    code = torch.stack((table[(c & 15).long()], table[(c >> 4).long()]), 2).view(rows, -1, 16)
    safe = sf[:, :, None].clamp(min=2.0 ** -9)
    q = (blocks / safe).clamp(-6, 6)
    step = torch.where(q.abs() < 2, 0.5, torch.where(q.abs() < 4, 1.0, 2.0))
    ok = (code - q).abs() <= step / 2 + 2 * err / safe + 2.0 ** -20 * q.abs()
    assert torch.all(torch.where(sf[:, :, None] > 0, ok, code == 0))


def test_nvfp4_feeds_the_product():
    M, N, K = 70, 264, 512
    x, r, w, b = problem(M, K, 5)
    _, _, wb, sfb = si.nvfp4_problem(9, M, N, K)
    n = g.layer_norm(dev(x), dev(w), dev(b), residual=dev(r), out="nvfp4")
    C = g.matmul_nvfp4(n.y, n.scales, wb.to(DEV), sfb.to(DEV))
    ref = torch.from_numpy(oracle.gemm_nvfp4(n.y.cpu(), n.scales.cpu(), wb, sfb))
    # one BF16 rounding, and FP32 accumulation over 512 products
    assert torch.all((C.cpu().double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-5 * ref.abs().max())


@pytest.mark.parametrize("out", ["bf16", "e4m3"])
def test_strides_and_offsets(out):
    """Columns of a wider matrix, at offsets that share and that do not share their misalignment."""
    rows, cols = 37, 1003
    for off_x, off_r, wide in ((0, 0, 1008), (3, 3, 1011), (1, 6, 1010), (8, 0, 1024)):
        x, r, w, b = problem(rows, cols, 11 * off_x + off_r)
        bx, br = (torch.full((rows, wide + 8), 9.0, dtype=BF16, device=DEV) for _ in range(2))
        vx, vr = bx[:, off_x:off_x + cols], br[:, off_r:off_r + cols]
        vx.copy_(x)
        vr.copy_(r)
        n = g.layer_norm(vx, dev(w), dev(b), residual=vr, out=out, inplace=True)
        d = Definition(x, r, w, b)
        assert n.sum.data_ptr() == vr.data_ptr() and torch.equal(vx.cpu(), x)
        outside = torch.ones(wide + 8, dtype=torch.bool)
        outside[off_r:off_r + cols] = False
        assert torch.all(br[:, outside.to(DEV)] == 9.0)
        d.check(n) if out == "bf16" else d.check_e4m3(n)


@pytest.mark.parametrize("cols", [264, 257])
def test_rows_with_zeros_infinities_and_nan(cols):
    x, _, w, b = problem(6, cols, 21, residual=False)
    x[1] = 0.0
    x[2, 5] = math.inf
    x[3, 7] = math.nan
    x[4, 3] = -math.inf
    n = g.layer_norm(dev(x), dev(w), dev(b), save=True)
    y = n.y.cpu()
    assert y[[2, 3, 4]].isnan().all()
    d = Definition(x[[0, 1, 5]], None, w, b)
    d.check_y(y[[0, 1, 5]])
    assert torch.equal(y[1], b)
    n = g.layer_norm(dev(x), dev(w), None, out="e4m3")
    sc = n.scales.cpu()
    assert sc[1] == 0 and torch.all(n.y[1].cpu().float() == 0)
    assert sc[[2, 3, 4]].isnan().all() and sc[[0, 5]].isfinite().all()
    assert not n.y.cpu().float()[[0, 1, 5]].isnan().any()


def backward_definition(dy, d, ds):
    g_ = dy.double()
    dyw = g_ * d.w
    c1, c2 = dyw.mean(1, keepdim=True), (dyw * d.xh).mean(1, keepdim=True)
    dx = d.rstd * (dyw - c1 - d.xh * c2) + (0 if ds is None else ds.double())
    # each term's size, and what xh's and rstd's errors move
    a1, a2 = dyw.abs().mean(1, keepdim=True), (dyw * d.xh).abs().mean(1, keepdim=True)
    size = d.rstd * (dyw.abs() + a1 + d.xh.abs() * a2) + (0 if ds is None else ds.double().abs())
    moved = d.rstd * (d.e_xh * a2 + d.xh.abs() * (dyw.abs() * d.e_xh).mean(1, keepdim=True)) + d.R * size
    return dx, moved + 2.0 ** -17 * size


def check_backward(dx, dw, db, dy, d, ds):
    want, tol = backward_definition(dy, d, ds)
    assert torch.all((dx.cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + 2 * tol)
    # rows are added within CTAs, then over at most 1216 CTAs in eight chains: fewer than 2^9 roundings deep here
    g_ = dy.double()
    assert torch.all((dw.cpu().double() - (g_ * d.xh).sum(0)).abs()
                     <= 2.0 ** -14 * (g_ * d.xh).abs().sum(0) + (g_.abs() * d.e_xh).sum(0) + 1e-30)
    assert torch.all((db.cpu().double() - g_.sum(0)).abs() <= 2.0 ** -14 * g_.abs().sum(0) + 1e-30)


@pytest.mark.parametrize("rows,cols", SHAPES + SEVERAL_ROWS)
@pytest.mark.parametrize("past", [True, False])
def test_backward(rows, cols, past):
    x, r, w, b = problem(rows, cols, 5 * rows + cols)
    dy = rand(rows, rows, cols)
    ds = rand(cols + 1, rows, cols, std=0.5) if past else None
    n = g.layer_norm(dev(x), dev(w), dev(b), residual=dev(r), eps=EPS, save=True)
    got = g.layer_norm_backward(dev(dy), n.sum, dev(w), n.mean, n.rstd, dsum=dev(ds))
    check_backward(*got, dy, Definition(x, r, w, b), ds)


def test_backward_against_differences():
    rows, cols = 2, 24
    x, _, w, b = problem(rows, cols, 77, residual=False)
    dy = rand(78, rows, cols)
    n = g.layer_norm(dev(x), dev(w), dev(b), save=True)
    dx, dw, db = g.layer_norm_backward(dev(dy), n.sum, dev(w), n.mean, n.rstd)

    def value(xd, wd, bd):
        var, mean = torch.var_mean(xd, 1, correction=0, keepdim=True)
        return (dy.double() * ((xd - mean) / (var + 1e-5).sqrt() * wd + bd)).sum()

    h, zero = 1e-5, torch.zeros(cols, dtype=torch.float64)
    at = (x.double(), w.double(), b.double())
    for i in range(rows):
        for j in range(0, cols, 5):
            e = torch.zeros(rows, cols, dtype=torch.float64)
            e[i, j] = h
            diff = (value(at[0] + e, *at[1:]) - value(at[0] - e, *at[1:])) / (2 * h)
            assert abs(dx[i, j].item() - diff.item()) <= 2.0 ** -8 * abs(diff.item()) + 1e-5
    for j in range(cols):
        e = zero.clone()
        e[j] = h
        for got, plus, minus in ((dw, (at[0], at[1] + e, at[2]), (at[0], at[1] - e, at[2])),
                                 (db, (at[0], at[1], at[2] + e), (at[0], at[1], at[2] - e))):
            diff = (value(*plus) - value(*minus)) / (2 * h)
            assert abs(got[j].item() - diff.item()) <= 1e-5 * (1 + abs(diff.item()))


def test_backward_repeats_bit_for_bit_in_place_and_in_part():
    rows, cols = 3001, 1027
    x, r, w, b = problem(rows, cols, 31)
    dy, ds = dev(rand(32, rows, cols)), dev(rand(33, rows, cols))
    n = g.layer_norm(dev(x), dev(w), dev(b), residual=dev(r), save=True)
    want = g.layer_norm_backward(dy, n.sum, dev(w), n.mean, n.rstd, dsum=ds)
    again = g.layer_norm_backward(dy, n.sum, dev(w), n.mean, n.rstd, dsum=ds)
    assert all(torch.equal(u, v) for u, v in zip(want, again))
    acc = ds.clone()
    g.gemm_layer_norm_backward(dy, n.sum, dev(w), n.mean, n.rstd, acc, acc, None, None, rows, cols)
    assert torch.equal(acc, want[0])
    db = torch.full((cols + 1,), 7.0, device=DEV)
    g.gemm_layer_norm_backward(dy, n.sum, dev(w), n.mean, n.rstd, ds, acc.clone(), None, db, rows, cols)
    assert torch.equal(db[:cols], want[2]) and db[cols] == 7
    none = g.layer_norm_backward(dy, n.sum, dev(w), n.mean, n.rstd, dsum=ds, weight_grads=False)
    assert torch.equal(none[0], want[0]) and none[1] is None and none[2] is None


@pytest.mark.parametrize("cols", [1003, 9001])
def test_several_rows_a_cta_that_share_no_alignment(cols):
    """x, the residual and the gradients at offsets and strides of their own: element by element."""
    rows = 1300
    x, r, w, b = problem(rows, cols, cols)
    dy, ds = rand(cols + 5, rows, cols), rand(cols + 6, rows, cols, std=0.5)

    def apart(t, before, wide):
        v = torch.full((rows, wide), 9.0, dtype=BF16, device=DEV)[:, before:before + cols]
        v.copy_(t)
        return v

    n = g.layer_norm(apart(x, 1, cols + 7), dev(w), dev(b), residual=apart(r, 6, cols + 9), eps=EPS, save=True)
    d = Definition(x, r, w, b)
    d.check(n)
    got = g.layer_norm_backward(apart(dy, 3, cols + 4), apart(d.s, 2, cols + 5), dev(w), n.mean, n.rstd,
                                dsum=apart(ds, 5, cols + 12))
    check_backward(*got, dy, d, ds)


def test_empty():
    w = torch.ones(16, dtype=BF16, device=DEV)
    n = g.layer_norm(torch.empty(0, 16, dtype=BF16, device=DEV), w, w, save=True)
    assert n.y.shape == (0, 16)
    _, dw, db = g.layer_norm_backward(torch.empty(0, 16, dtype=BF16, device=DEV), n.sum, w, n.mean, n.rstd)
    assert torch.all(dw == 0) and torch.all(db == 0)
    x = torch.empty(300, 0, dtype=BF16, device=DEV)
    n = g.layer_norm(x, save=True, out="e4m3")
    assert torch.all(n.mean == 0) and torch.all(n.rstd == 0) and torch.all(n.scales == 0)
    dx, dw, db = g.layer_norm_backward(x, n.sum, None, n.mean, n.rstd)
    assert dx.shape == (300, 0) and dw.shape == (0,) and db.shape == (0,)


def test_graph_capture():
    x, r, w, b = (dev(t) for t in problem(400, 1040, 51))
    dy = dev(rand(52, 400, 1040))

    def step():
        m = g.layer_norm(x, w, b, residual=r, save=True)
        return (m.y, *g.layer_norm_backward(dy, m.sum, w, m.mean, m.rstd))

    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want))


# nine, sixteen and seventeen warps with the last at a row's ends; two, three and four groups a thread on either side of
# where they begin
@pytest.mark.parametrize("cols", [4095, 4097, 4604, 4617, 7675, 7693, 8190, 8192, 8193, 8200, 10001, 11527, 11530, 12288, 12290,
                                  12296])
@pytest.mark.parametrize("own", [False, True])
def test_backward_around_the_shapes(cols, own):
    """`own`: rows whose tensors lie differently against the 16-byte boundary."""
    rows = 330
    x, r, w, b = problem(rows, cols, cols)
    dy, ds = rand(5, rows, cols), rand(6, rows, cols, std=0.5)
    n = g.layer_norm(dev(x), dev(w), dev(b), residual=dev(r), eps=EPS, save=True)
    put = dev(dy)
    if own:
        put = torch.empty(rows, cols + 5, dtype=BF16, device=DEV)[:, 3:cols + 3]
        put.copy_(dy)
    check_backward(*g.layer_norm_backward(put, n.sum, dev(w), n.mean, n.rstd, dsum=dev(ds)), dy, Definition(x, r, w, b), ds)


class OnTheDevice(Definition):
    """The same, computed where the rows are (the CPU takes a minute for these)."""

    def __init__(self, x, r, w, b):
        with torch.device(DEV):
            super().__init__(x, r, w, b)


# with a residual to BF16 on the 16-byte boundary, 16 bytes for each of rows x cols elements of more than 1.5 times L2: fewer
# rows on their way, two of them ahead from 4096 columns on, by a limit through shared memory; widths of whole and of ragged
# warps, one to eight CTAs an SM
@pytest.mark.parametrize("rows,cols", [(8192, 4096), (9000, 3080), (3301, 8192), (24001, 1160), (33000, 776), (6100, 4488)])
def test_four_streams_past_l2(rows, cols):
    assert 16 * rows * cols > 3 * torch.cuda.get_device_properties(DEV).L2_cache_size and 96 * 8 < cols <= 8192
    gen = torch.Generator(device=DEV).manual_seed(cols)
    x, r = (torch.randn(rows, cols, generator=gen, device=DEV).to(BF16) for _ in range(2))
    _, _, w, b = problem(1, cols, 5)
    w, b = dev(w), dev(b)
    n = g.layer_norm(x, w, b, residual=r, eps=EPS, save=True)
    d = OnTheDevice(x, r, w, b)
    assert torch.equal(n.sum, d.s)
    assert torch.all((n.mean.double()[:, None] - d.mean).abs() <= d.e)
    assert torch.all((n.rstd.double()[:, None] - d.rstd).abs() <= d.R * d.rstd)
    assert torch.all((n.y.double() - d.y).abs() <= 2.0 ** -8 * d.y.abs() + 2 * d.err)
    stream = r.clone()
    again = g.layer_norm(x, w, b, residual=stream, eps=EPS, save=True, inplace=True)
    assert again.sum.data_ptr() == stream.data_ptr()
    assert all(torch.equal(u, v) for u, v in zip((n.y, n.sum, n.mean, n.rstd), (again.y, stream, again.mean, again.rstd)))


# rows enough for several a CTA, off the boundary with 8 to 11 and 17 warps (the last one with a row's ends) and three and four
# groups a thread, on it with four
@pytest.mark.parametrize("rows,cols", [(700, 4087), (700, 4099), (700, 4401), (700, 4701), (500, 8195), (400, 10003), (330, 14003),
                                       (330, 16008), (330, 15366)])
def test_rows_of_many_warps(rows, cols):
    x, r, w, b = problem(rows, cols, cols)
    d = Definition(x, r, w, b)
    n = g.layer_norm(dev(x), dev(w), dev(b), residual=dev(r), eps=EPS, save=True)
    d.check(n)
    d.check_e4m3(g.layer_norm(dev(x), dev(w), dev(b), residual=dev(r), eps=EPS, out="e4m3"))
    dy, ds = rand(rows, rows, cols), rand(cols + 1, rows, cols, std=0.5)
    got = g.layer_norm_backward(dev(dy), n.sum, dev(w), n.mean, n.rstd, dsum=dev(ds))
    check_backward(*got, dy, d, ds)


@pytest.mark.parametrize("cols", [16, 200, 255, 256, 257, 1024, 1025, 4099, 20000, 20001])
@pytest.mark.parametrize("rows", [7, 700])
def test_sums_past_fp32_make_the_row_nan_at_every_width(cols, rows):
    """2^70 squared passes FP32's range: such a row counts as one with an infinity, whether a warp has it alone or not, and its
    statistics are NaN as its other outputs."""
    x = rand(cols, rows, cols).to(DEV)
    at = torch.arange(cols, device=DEV)
    x[1] = torch.where(at % 2 == 0, 2.0 ** 70, -(2.0 ** 70)).to(BF16)
    x[2, cols // 2] = math.inf
    x[3, 0] = -math.inf
    x[4, cols - 1] = math.nan
    x[5] = torch.where(at % 2 == 0, 2.0 ** 50, -(2.0 ** 50)).to(BF16)  # (squares that FP32 holds)
    bad = torch.zeros(rows, dtype=torch.bool, device=DEV)
    bad[1:5] = True
    w, b = (t.to(DEV) for t in problem(1, cols, 3)[2:])
    n = g.layer_norm(x, w, b, save=True)
    for t in (n.mean, n.rstd, n.y[:, 0], n.y[:, -1]):
        assert torch.equal(t.isnan(), bad)
    assert n.y[1:5].isnan().all() and not n.y[5:].isnan().any()
    n = g.layer_norm(x, w, b, out="e4m3")
    assert torch.equal(n.scales.isnan(), bad) and n.y[1:5].float().isnan().all() and not n.y[5:].float().isnan().any()
    if cols % 16 == 0:
        n = g.layer_norm(x, w, b, out="nvfp4")
        assert torch.equal(n.scales.view(torch.float8_e4m3fn).float().isnan().all(1), bad)
