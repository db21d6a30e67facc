"""gemm_embedding and its gradient through the binding, against FP64 evaluations of their definitions.

Tolerances, derived before the first run. A looked-up value is one FP32 product rounded once: off by 2^-24 and, in BF16,
2^-8 of itself. A token's sum of n rows goes through at most n FP32 additions, each off by 2^-24 of a partial sum that is no
larger than the sum of magnitudes: n 2^-24 of that; scale and base add two roundings, the output 2^-8 (BF16) or 2^-24.
"""
import pytest
import torch

import dense_tensor_core_persistent_gb300 as g
from dense_tensor_core_persistent_gb300 import build as gbuild

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gbuild.build()


def normal(seed, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def ids(seed, n, vocab, kind="uniform"):
    gen = torch.Generator().manual_seed(seed)
    t = torch.randint(0, vocab, (n,), generator=gen)
    if kind == "one":
        t[:] = vocab - 1
    elif kind == "few":
        t = t % 3 * (vocab // 3)
    elif kind == "frequent":
        t = torch.where(torch.rand(n, generator=gen) < 0.3, vocab // 2, t)
    if n > 4 and kind != "one":
        t[torch.rand(n, generator=gen) < 0.1] = -1
    return t.to(DEV)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab,cols", [(1, 1, 1), (1, 1000, 8192), (5, 7, 3), (64, 5000, 520), (33, 100, 1027),
                                             (3000, 300, 64), (700, 2000, 4104), (2, 9, 9000)])
@pytest.mark.parametrize("scale", [1.0, 11.3])
def test_lookup(dtype, rows, vocab, cols, scale):
    table, tokens = normal(rows, vocab, cols, dtype=dtype), ids(cols, rows, vocab)
    y = g.embedding(table, tokens, scale=scale)
    want = table.double()[tokens.clamp(min=0)] * scale * (tokens >= 0)[:, None]
    assert y.dtype == dtype and y.shape == (rows, cols)
    assert torch.all((y.double() - want).abs() <= (HALF_STEP[dtype] + 2.0 ** -22) * want.abs())
    if scale == 1.0:
        assert torch.equal(y.double(), want)


@pytest.mark.parametrize("dtype", TYPES)
def test_lookup_strides_and_tokens_outside(dtype):
    vocab, cols = 50, 72
    wide = normal(1, vocab, cols + 11, dtype=dtype)
    tokens = torch.tensor([3, -1, 50, 49, -(1 << 40), 1 << 40, 0], device=DEV)
    for off in (0, 3, 8):
        view = wide[:, off:off + cols]
        y = g.embedding(view, tokens)
        assert torch.equal(y[[0, 3, 6]], view[[3, 49, 0]])
        assert torch.all(y[[1, 4]] == 0) and y[[2, 5]].isnan().all()
    out = torch.full((9, cols + 5), 7.0, dtype=dtype, device=DEV)
    g.gemm_embedding(wide, g._table_kind(dtype, ""), tokens, out, 7, vocab, cols, cols + 11, cols + 5)
    assert torch.equal(out[0, :cols], wide[3, :cols]) and torch.all(out[:, cols:] == 7) and torch.all(out[7:] == 7)
    assert g.embedding(wide, tokens[:0]).shape == (0, cols + 11)


def check_gradient(got, dy, tokens, vocab, scale, base):
    ok = (tokens >= 0) & (tokens < vocab)
    at, rows = tokens[ok], dy[ok].double()
    want = torch.zeros(vocab, dy.shape[1], dtype=torch.float64, device=DEV) if base is None else base.double()
    size = want.abs()
    want = want.index_put((at,), rows * scale, accumulate=True)
    size = size.index_put((at,), rows.abs() * scale, accumulate=True)
    n = torch.bincount(at, minlength=vocab)[:, None].double() + 3
    tol = n * 2.0 ** -24 * size
    assert torch.all((got.double() - want).abs() <= tol + HALF_STEP[got.dtype] * (want.abs() + tol))
    untouched = n[:, 0] == 3
    assert torch.equal(got[untouched], torch.zeros_like(got[untouched]) if base is None else base[untouched])


@pytest.mark.parametrize("kind", ["uniform", "one", "few", "frequent"])
@pytest.mark.parametrize("rows,vocab,cols", [(1, 1, 1), (1, 300, 64), (17, 40, 8), (300, 513, 1027), (2000, 70000, 136),
                                             (9001, 262143, 24), (5000, 3000, 2056), (30000, 262145, 16)])
def test_gradient(kind, rows, vocab, cols):
    dy, tokens = normal(rows, rows, cols), ids(vocab, rows, vocab, kind)
    check_gradient(g.embedding_backward(dy, tokens, vocab, scale=1.5), dy, tokens, vocab, 1.5, None)


@pytest.mark.parametrize("dy_type", TYPES)
@pytest.mark.parametrize("out_type", TYPES)
@pytest.mark.parametrize("rows,vocab,cols", [(300, 257, 64), (1500, 1000, 1003), (77, 5001, 4)])
def test_types_base_and_in_place(dy_type, out_type, rows, vocab, cols):
    dy, tokens = normal(2, rows, cols, dtype=dy_type), ids(3, rows, vocab, "frequent")
    base = normal(4, vocab, cols, dtype=out_type)
    got = g.embedding_backward(dy, tokens, vocab, scale=0.7, base=base)
    assert got.dtype == out_type
    check_gradient(got, dy, tokens, vocab, 0.7, base)
    check_gradient(g.embedding_backward(dy, tokens, vocab, dtype=out_type), dy, tokens, vocab, 1.0, None)
    mine = base.clone()
    out = g.embedding_backward(dy, tokens, vocab, scale=0.7, base=mine, inplace=True)
    assert out.data_ptr() == mine.data_ptr() and torch.equal(out, got)


def test_what_is_not_read_and_not_written():
    """Rows of NaN at places without a token, a gradient with strides, memory around the table."""
    rows, vocab, cols = 400, 60, 40
    tokens = ids(5, rows, vocab)
    tokens[3], tokens[7] = vocab, 1 << 50
    wide = torch.full((rows, cols + 9), float("nan"), dtype=torch.bfloat16, device=DEV)
    dy = normal(6, rows, cols)
    wide[:, 1:cols + 1] = dy
    outside = (tokens < 0) | (tokens >= vocab)
    wide[outside] = float("nan")
    check_gradient(g.embedding_backward(wide[:, 1:cols + 1], tokens, vocab), dy, tokens, vocab, 1.0, None)
    buf = torch.full((vocab + 2, cols), 7.0, dtype=torch.bfloat16, device=DEV)
    g.gemm_embedding_backward(dy, g.GEMM_TABLE_BF16, tokens, None, buf, g.GEMM_TABLE_BF16, rows, vocab, cols)
    assert torch.all(buf[vocab:] == 7)
    # in place at an odd offset
    flat = torch.full((vocab * cols + 9,), 7.0, dtype=torch.bfloat16, device=DEV)
    table = flat[1:1 + vocab * cols].view(vocab, cols)
    table.fill_(0.5)
    base = table.clone()
    got = g.embedding_backward(dy, tokens, vocab, base=table, inplace=True)
    check_gradient(got, dy, tokens, vocab, 1.0, base)
    assert flat[0] == 7 and torch.all(flat[1 + vocab * cols:] == 7)


def test_no_positions():
    dy, tokens = normal(1, 0, 24), torch.empty(0, dtype=torch.int64, device=DEV)
    assert torch.all(g.embedding_backward(dy, tokens, 33) == 0)
    base = normal(2, 33, 24)
    assert torch.equal(g.embedding_backward(dy, tokens, 33, base=base), base)
    assert torch.equal(g.embedding_backward(dy, tokens, 33, base=base, inplace=True), base)
    none = torch.full((5,), -1, device=DEV)
    assert torch.all(g.embedding_backward(normal(3, 5, 24), none, 33) == 0)


def test_order_of_positions_and_repeats():
    """Two positions of a token add in their order whatever stands between them, bit for bit each time."""
    rows, vocab, cols = 60000, 50, 64
    tokens = ids(9, rows, vocab, "frequent")
    dy = normal(10, rows, cols, dtype=torch.float32)
    a = g.embedding_backward(dy, tokens, vocab)
    check_gradient(a, dy, tokens, vocab, 1.0, None)
    assert all(torch.equal(a, g.embedding_backward(dy, tokens, vocab)) for _ in range(3))
    # 1e8 and -1e8 cancel before the small one comes; in another order it would be lost
    dy = torch.zeros(200, 8, device=DEV)
    tokens = torch.full((200,), 5, device=DEV)
    tokens[100:103] = 7
    dy[100], dy[101], dy[102] = 1e8, -1e8, 0.25
    assert torch.all(g.embedding_backward(dy, tokens, 9)[7] == 0.25)


def test_against_differences():
    """The gradient of sum(dy * embedding(table)) by differences of the lookup itself, which is linear."""
    vocab, cols, rows = 6, 8, 20
    table, tokens, dy = normal(1, vocab, cols, dtype=torch.float32), ids(2, rows, vocab), normal(3, rows, cols,
                                                                                              dtype=torch.float32)
    grad = g.embedding_backward(dy, tokens, vocab, scale=3.0)
    for v in range(vocab):
        for c in range(0, cols, 3):
            up, down = table.clone(), table.clone()
            up[v, c] += 0.5
            down[v, c] -= 0.5
            diff = ((g.embedding(up, tokens, scale=3.0).double() - g.embedding(down, tokens, scale=3.0).double())
                    * dy.double()).sum()
            assert abs(diff.item() - grad[v, c].item()) <= 2.0 ** -18 * rows * 3 * 4


def test_captured_and_replayed():
    vocab, cols, rows = 3000, 136, 900
    table, dy = normal(1, vocab, cols), normal(2, rows, cols)
    tokens, other = ids(3, rows, vocab), ids(4, rows, vocab, "frequent")

    def step(t):
        return g.embedding(table, t), g.embedding_backward(dy, t, vocab)

    want = step(other)
    static = tokens.clone()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(static)
        graphs.append((graph, out))
    static.copy_(other)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(u, v) for u, v in zip(out, want))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", [8, 5])
def test_lengths_around_the_runs(dtype, cols):
    """Tokens of 1 to 70 positions one behind the other, from every offset against the runs of positions: short ones that
    cross a run's end, long ones that begin, cross and end anywhere, and places without a token behind them."""
    for lead in range(0, 40, 3):
        lengths = [lead] + [1, 31, 2, 32, 33, 1, 1, 34, 64, 7, 8, 9, 65, 3, 70, 40, 15, 16, 17, 36]
        tokens = torch.cat([torch.full((n,), 2 * v) for v, n in enumerate(lengths)] + [torch.full((lead,), -1)])
        order = torch.randperm(len(tokens), generator=torch.Generator().manual_seed(lead))
        tokens = tokens[order].to(DEV)
        dy = normal(lead, len(tokens), cols, dtype=dtype)
        check_gradient(g.embedding_backward(dy, tokens, 43, scale=0.5), dy, tokens, 43, 0.5, None)


def test_many_positions_of_few_tokens():
    """Runs of more than the least length, and long tokens of thousands of runs."""
    for rows, vocab in ((100000, 3), (70000, 1), (300001, 70000)):
        tokens, dy = ids(rows, rows, vocab, "few" if vocab == 3 else "frequent"), normal(7, rows, 8)
        check_gradient(g.embedding_backward(dy, tokens, vocab), dy, tokens, vocab, 1.0, None)


@pytest.mark.parametrize("rows,vocab", [(16384, 1025), (16385, 1 << 20), (131072, 1 << 10), (131073, 5000), (257, (1 << 21) + 3),
                                        (40000, (1 << 21) + 3)])
def test_sorts_of_every_kind(rows, vocab):
    """Around the lengths from which the sort takes more CTAs and reads its entries again, in one to three passes."""
    tokens, dy = ids(rows, rows, vocab, "frequent"), normal(rows, rows, 4)
    check_gradient(g.embedding_backward(dy, tokens, vocab), dy, tokens, vocab, 1.0, None)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab,cols", [(16384, 3000, 4096), (1301, 70000, 4104), (1400, 900, 4099), (9000, 500, 1027),
                                             (700001, 100, 8), (700001, 100, 7)])
def test_lookup_of_many_rows(dtype, rows, vocab, cols):
    """Rows and vectors enough for four loads a thread in flight."""
    assert rows * -(-cols // 8) >= 4096 * torch.cuda.get_device_properties(DEV).multi_processor_count
    gen = torch.Generator(device=DEV).manual_seed(cols)
    table = torch.randn(vocab, cols + 8, generator=gen, device=DEV).to(dtype)[:, :cols]
    tokens = torch.randint(0, vocab, (rows,), generator=gen, device=DEV)
    tokens[torch.rand(rows, generator=gen, device=DEV) < 0.1] = -5
    tokens[rows // 2] = vocab
    want = torch.where((tokens >= 0)[:, None], table[tokens.clamp(0, vocab - 1)], 0.0)
    want[rows // 2] = float("nan")
    y = g.embedding(table, tokens)
    assert torch.equal(y.nan_to_num(7.0), want.nan_to_num(7.0))
    out = torch.full((rows + 1, cols + 8), 7.0, dtype=dtype, device=DEV)
    g.gemm_embedding(table, g._table_kind(dtype, ""), tokens, out, rows, vocab, cols, cols + 8, cols + 8)
    assert torch.equal(out[:rows, :cols].nan_to_num(7.0), want.nan_to_num(7.0))
    assert torch.all(out[:, cols:] == 7) and torch.all(out[rows] == 7)


@pytest.mark.parametrize("rows", [257, 4000, 16384, 20000, 131073, 200000])
@pytest.mark.parametrize("dtype", TYPES)
def test_order_of_positions_through_the_sort(rows, dtype):
    """As test_order_of_positions_and_repeats where positions are sorted: by 8 CTAs, by 16 (above 16384 positions), and with its
    entries read again (above 131072). Three positions of a token a long way apart, in their order within one warp's part of
    the list, in two warps' and in two CTAs', cancel before the small one comes, which any other order would lose; the short
    tokens stand beside one another and beside a long one in the sorted list."""
    vocab, cols = 5000, 8
    gen = torch.Generator().manual_seed(rows)
    tokens = torch.randint(0, 100, (rows,), generator=gen)  # (long ones, none above 99)
    tokens[torch.rand(rows, generator=gen) < 0.1] = -1
    dy = torch.zeros(rows, cols)
    places = torch.randperm(rows, generator=gen)[:240].view(80, 3).sort(1).values
    places[0] = torch.tensor([0, rows // 2, rows - 1])
    places[1] = torch.tensor([1, 2, 3])
    places[2] = torch.tensor([31, 32, 33])
    places[3] = torch.tensor([63, 64, 255])
    kept = torch.ones(80, dtype=torch.bool)
    seen = set()
    for i in range(80):  # (random ones that took another's place are left out)
        if seen & set(places[i].tolist()):
            kept[i] = False
        else:
            seen |= set(places[i].tolist())
    places = places[kept]
    ids = 1000 + 7 * torch.arange(len(places))
    for i, (a, b, c) in enumerate(places.tolist()):
        tokens[a] = tokens[b] = tokens[c] = ids[i]
        dy[a], dy[b], dy[c] = 2.0 ** 27, -2.0 ** 27, 0.25
    got = g.embedding_backward(dy.to(dtype).to(DEV), tokens.to(DEV), vocab)
    assert torch.all(got[ids.to(DEV)] == 0.25)
    # one token of 16 positions, the most that are added one after the other, within a run of sorted positions or across two
    for lead in range(8):
        tokens[:] = -1
        tokens[:lead] = 1
        at = torch.randperm(rows - lead, generator=gen)[:16].sort().values + lead
        tokens[at] = 2
        dy[:] = 0
        for i in range(15):
            dy[at[i]] = 2.0 ** 27 * (-1) ** i if i < 14 else 0.25
        dy[at[15]] = 0.5
        got = g.embedding_backward(dy.to(dtype).to(DEV), tokens.to(DEV), vocab)
        assert torch.all(got[2] == 0.75)


@pytest.mark.parametrize("dtype", TYPES)
def test_a_base_that_is_written_again_between_two_calls(dtype):
    """By a copy from the host, which no SM sees, right after kernels have read it: what they left in an L1 must not be read
    again by the kernel that copies the base beside the sort."""
    for vocab in (1000, 20000):
        cols, rows = 1024, 300
        base = torch.zeros(vocab, cols, dtype=dtype, device=DEV)
        tokens, dy = ids(1, rows, vocab), torch.zeros(rows, cols, dtype=dtype, device=DEV)
        host = [torch.full((vocab, cols), float(v), dtype=dtype).pin_memory() for v in (1, 2)]
        for i in range(10):
            g.embedding_backward(dy, tokens, vocab, base=base)
            base.copy_(host[i % 2], non_blocking=True)
            assert torch.all(g.embedding_backward(dy, tokens, vocab, base=base) == 1 + i % 2)
