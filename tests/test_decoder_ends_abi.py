"""Argument checks of the operators at a decoder's ends (no GPU needed: refusals come before any device use)."""
import pytest
import torch

import dense_tensor_core_persistent_gb300 as g
from dense_tensor_core_persistent_gb300 import build as gbuild

BAD, SHAPE, ALIGN = g.GEMM_ERR_INVALID_ARG, g.GEMM_ERR_UNSUPPORTED_SHAPE, g.GEMM_ERR_MISALIGNED


@pytest.fixture(scope="module", autouse=True)
def built():
    gbuild.build()


def loss(x=16, w=16, t=16, loss=16, lse=16, M=2, V=5, K=8, scale=1.0, strides=None):
    return g.lib().gemm_cross_entropy(x, w, t, loss, lse, M, V, K, scale, 0, strides)


def loss_backward(x=16, w=16, t=16, lse=16, dloss=16, dlse=16, dx=16, dw=16, M=2, V=5, K=8, scale=1.0, ws=0, strides=None):
    return g.lib().gemm_cross_entropy_backward(x, w, t, lse, dloss, dlse, dx, dw, M, V, K, scale, ws, 0, strides)


def test_cross_entropy_refusals():
    assert loss(M=0, x=0, w=0, lse=0) == g.GEMM_OK
    assert loss(M=-1) == BAD and loss(V=-1) == BAD and loss(K=-8) == BAD and loss(V=0) == BAD
    assert loss(x=0) == BAD and loss(w=0) == BAD and loss(lse=0) == BAD
    assert loss(t=0) == BAD and loss(loss=0) == BAD  # one without the other
    assert loss(K=12) == SHAPE
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert loss(scale=scale) == BAD
    assert loss(x=24) == ALIGN and loss(w=8) == ALIGN and loss(t=20) == ALIGN and loss(lse=18) == ALIGN
    assert loss(strides=g.gemm_cross_entropy_strides_t(4, 0)) == BAD
    assert loss(strides=g.gemm_cross_entropy_strides_t(12, 0)) == SHAPE


def test_cross_entropy_backward_refusals():
    assert loss_backward(dx=0, dw=0) == g.GEMM_OK  # nothing asked for
    assert loss_backward(M=0, dw=0) == g.GEMM_OK and loss_backward(K=0) == g.GEMM_OK
    assert loss_backward(M=-1) == BAD and loss_backward(V=-1) == BAD and loss_backward(V=0) == BAD
    assert loss_backward(t=0) == BAD and loss_backward(dloss=0) == BAD  # one without the other
    assert loss_backward(x=0) == BAD and loss_backward(w=0) == BAD and loss_backward(lse=0) == BAD
    assert loss_backward(K=4) == SHAPE and loss_backward(scale=0.0) == BAD
    assert loss_backward(strides=g.gemm_cross_entropy_strides_t(0, 12)) == SHAPE
    assert loss_backward(strides=g.gemm_cross_entropy_strides_t(0, 4)) == BAD
    assert loss_backward(dx=8) == ALIGN and loss_backward(dw=8) == ALIGN and loss_backward(dlse=18) == ALIGN
    assert loss_backward(dloss=17) == ALIGN and loss_backward(t=20) == ALIGN


def test_cross_entropy_piece():
    assert g.cross_entropy_piece(4096, 50000) == 50000  # G fits
    assert g.cross_entropy_piece(4096, 131072) == 65536
    assert g.cross_entropy_piece(1, 131072) == 131072 and g.cross_entropy_piece(0, 7) == 7
    assert g.cross_entropy_piece(1 << 20, 131072) == 256  # never less than a tile
    for M, V, ws in ((300, 8005, 2 * 300 * 1000), (7, 3000, 1), (5000, 262144, 1 << 27)):
        piece = g.cross_entropy_piece(M, V, ws)
        assert piece % 256 == 0 and (piece == 256 or 2 * M * piece <= ws)
    for bad in ((-1, 5), (5, -1)):
        with pytest.raises(g.GemmError):
            g.cross_entropy_piece(*bad)


def test_binding_refuses_tensors_that_are_not_what_it_takes():
    x = torch.zeros(2, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x:"):
        g.cross_entropy(x, x)  # not on a GPU
    with pytest.raises(ValueError, match="x:"):
        g.cross_entropy(None, x)
    with pytest.raises(ValueError, match="x:"):
        g.cross_entropy_backward(None, x, None, None, None)


def test_no_device_is_reported():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert loss() == g.GEMM_ERR_NO_DEVICE
    assert loss_backward() == g.GEMM_ERR_NO_DEVICE


def norm(x=16, r=0, w=16, b=16, s=0, y=16, scales=0, mean=0, rstd=0, rows=2, cols=32, eps=1e-5, fmt=0, strides=None):
    return g.lib().gemm_layer_norm(x, r, w, b, s, y, scales, mean, rstd, rows, cols, eps, fmt, 0, strides)


def norm_backward(dy=16, s=16, w=16, mean=16, rstd=16, ds=0, dx=16, dw=16, db=16, rows=2, cols=32, strides=None):
    return g.lib().gemm_layer_norm_backward(dy, s, w, mean, rstd, ds, dx, dw, db, rows, cols, 0, strides)


def test_layer_norm_refusals():
    assert norm(rows=0, x=0, y=0) == g.GEMM_OK and norm(cols=0, x=0, y=0) == g.GEMM_OK
    assert norm(rows=-1) == BAD and norm(cols=-1) == BAD
    assert norm(eps=-1.0) == BAD and norm(eps=float("nan")) == BAD
    assert norm(fmt=3) == BAD and norm(fmt=-1) == BAD
    assert norm(x=0) == BAD and norm(y=0) == BAD
    assert norm(fmt=g.GEMM_NORM_E4M3) == BAD  # no scales
    assert norm(r=16, s=0) == BAD  # the sum has nowhere to go
    assert norm(cols=32761) == SHAPE
    assert norm(fmt=g.GEMM_NORM_NVFP4, scales=16, cols=24) == SHAPE
    assert norm(fmt=g.GEMM_NORM_NVFP4, scales=16, x=18) == ALIGN and norm(fmt=g.GEMM_NORM_NVFP4, scales=16, b=18) == ALIGN
    assert norm(x=17) == ALIGN and norm(b=17) == ALIGN and norm(mean=18) == ALIGN and norm(rstd=18) == ALIGN
    assert norm(cols=0, mean=18) == ALIGN
    assert norm(strides=g.gemm_norm_strides_t(31, 0, 0, 0)) == BAD
    assert norm(fmt=g.GEMM_NORM_NVFP4, scales=16, strides=g.gemm_norm_strides_t(0, 0, 0, 48)) == SHAPE


def test_layer_norm_backward_refusals():
    assert norm_backward(cols=0, dy=0) == g.GEMM_OK
    assert norm_backward(rows=0, dy=0, s=0, mean=0, rstd=0, dx=0, dw=0, db=0) == g.GEMM_OK
    assert norm_backward(rows=-1) == BAD and norm_backward(cols=-3) == BAD
    assert norm_backward(dy=0) == BAD and norm_backward(s=0) == BAD and norm_backward(dx=0) == BAD
    assert norm_backward(mean=0) == BAD and norm_backward(rstd=0) == BAD
    assert norm_backward(cols=32761) == SHAPE
    assert norm_backward(dx=17) == ALIGN and norm_backward(dw=18) == ALIGN and norm_backward(db=18) == ALIGN
    assert norm_backward(strides=g.gemm_norm_backward_strides_t(0, 0, 8, 0)) == BAD


def test_layer_norm_binding_refuses():
    x = torch.zeros(2, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x:"):
        g.layer_norm(x)
    with pytest.raises(ValueError, match="out:"):
        g.layer_norm(x, out="int8")
    with pytest.raises(ValueError, match="total:"):
        g.layer_norm_backward(x, x, None, None, None)


def test_layer_norm_without_a_device():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert norm() == g.GEMM_ERR_NO_DEVICE
    assert norm_backward() == g.GEMM_ERR_NO_DEVICE


def lookup(table=16, kind=0, tokens=16, y=16, rows=2, vocab=5, cols=8, ldt=0, ldy=0, scale=1.0):
    return g.lib().gemm_embedding(table, kind, tokens, y, rows, vocab, cols, ldt, ldy, scale, 0)


def table_grad(dy=16, dk=0, tokens=16, base=0, out=16, tk=0, rows=2, vocab=5, cols=8, ldd=0, scale=1.0):
    return g.lib().gemm_embedding_backward(dy, dk, tokens, base, out, tk, rows, vocab, cols, ldd, scale, 0)


def test_embedding_refusals():
    assert lookup(rows=0, table=0) == g.GEMM_OK and lookup(cols=0) == g.GEMM_OK
    assert lookup(rows=-1) == BAD and lookup(vocab=-1) == BAD and lookup(cols=-1) == BAD and lookup(kind=2) == BAD
    assert lookup(table=0) == BAD and lookup(tokens=0) == BAD and lookup(y=0) == BAD
    assert lookup(ldt=7) == BAD and lookup(ldy=-1) == BAD
    assert lookup(scale=float("inf")) == BAD and lookup(scale=float("nan")) == BAD
    assert lookup(cols=(1 << 22) + 1) == SHAPE
    assert lookup(table=17) == ALIGN and lookup(kind=1, y=18) == ALIGN and lookup(tokens=20) == ALIGN


def test_embedding_backward_refusals():
    assert table_grad(vocab=0, out=0) == g.GEMM_OK and table_grad(cols=0) == g.GEMM_OK
    assert table_grad(rows=0, base=16, out=16, dy=0) == g.GEMM_OK  # in place, and nothing to add
    assert table_grad(rows=-1) == BAD and table_grad(vocab=-1) == BAD and table_grad(dk=2) == BAD and table_grad(tk=-1) == BAD
    assert table_grad(dy=0) == BAD and table_grad(tokens=0) == BAD and table_grad(out=0) == BAD
    assert table_grad(ldd=7) == BAD and table_grad(scale=float("nan")) == BAD
    assert table_grad(vocab=1 << 27) == SHAPE and table_grad(cols=(1 << 22) + 1) == SHAPE
    assert table_grad(dy=17) == ALIGN and table_grad(tokens=4) == ALIGN and table_grad(out=24) == ALIGN
    assert table_grad(base=24, out=32) == ALIGN and table_grad(base=17, out=17) == ALIGN


def test_embedding_binding_refuses():
    x = torch.zeros(2, 32, dtype=torch.bfloat16)
    ids = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="table:"):
        g.embedding(x, ids)  # not on a GPU
    with pytest.raises(ValueError, match="table:"):
        g.embedding(x.half(), ids)
    with pytest.raises(ValueError, match="dy:"):
        g.embedding_backward(x, ids, 4)
    with pytest.raises(ValueError, match="table:"):
        g.embedding(None, ids)


def test_embedding_without_a_device():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert lookup() == g.GEMM_ERR_NO_DEVICE
    assert table_grad() == g.GEMM_ERR_NO_DEVICE


class OnDevice:
    """As much of a CUDA tensor as the binding's checks look at."""

    def __init__(self, index, dtype, shape):
        self.index, self.dtype, self.shape, self.is_cuda, self.device = index, dtype, torch.Size(shape), True, f"cuda:{index}"

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True


def test_tensors_of_another_device_are_refused(monkeypatch):
    monkeypatch.setattr(g, "_device", lambda: 0)
    bf16, i64 = torch.bfloat16, torch.int64
    with pytest.raises(ValueError, match="x: lies on cuda:1"):
        g.cross_entropy(OnDevice(1, bf16, (2, 8)), OnDevice(0, bf16, (5, 8)))
    with pytest.raises(ValueError, match="head: lies on cuda:1"):
        g.cross_entropy(OnDevice(0, bf16, (2, 8)), OnDevice(1, bf16, (5, 8)))
    with pytest.raises(ValueError, match="tokens: lies on cuda:2"):
        g.embedding(OnDevice(0, bf16, (5, 8)), OnDeviceVector(2, i64, 3))
    with pytest.raises(ValueError, match="bias: lies on cuda:1"):
        x = OnDevice(0, bf16, (2, 8))
        g.layer_norm(x, None, OnDeviceVector(1, bf16, 8))


class OnDeviceVector(OnDevice):
    def __init__(self, index, dtype, n):
        super().__init__(index, dtype, (n,))

    def numel(self):
        return self.shape[0]


def test_sizes_that_do_not_belong_together_are_refused(monkeypatch):
    monkeypatch.setattr(g, "_device", lambda: 0)
    bf16, f32, i64 = torch.bfloat16, torch.float32, torch.int64
    x, head = OnDevice(0, bf16, (2, 8)), OnDevice(0, bf16, (5, 8))
    with pytest.raises(ValueError, match="head: rows of 8"):
        g.cross_entropy(x, OnDevice(0, bf16, (5, 16)))
    with pytest.raises(ValueError, match="targets:"):
        g.cross_entropy(x, head, OnDeviceVector(0, i64, 3))
    with pytest.raises(ValueError, match="targets:"):
        g.cross_entropy(x, head, OnDeviceVector(0, torch.int32, 2))
    with pytest.raises(ValueError, match="lse:"):
        g.cross_entropy_backward(x, head, None, OnDeviceVector(0, f32, 3), None)
    with pytest.raises(ValueError, match="workspace:"):
        g.cross_entropy_backward(x, head, None, OnDeviceVector(0, f32, 2), None, workspace=-1)
    with pytest.raises(ValueError, match="inplace:"):
        g.embedding_backward(x, OnDeviceVector(0, i64, 2), 5, inplace=True)
    with pytest.raises(ValueError, match="base:"):
        g.embedding_backward(x, OnDeviceVector(0, i64, 2), 5, base=OnDevice(0, bf16, (4, 8)))
    with pytest.raises(ValueError, match="dtype:"):
        g.embedding_backward(x, OnDeviceVector(0, i64, 2), 5, dtype=torch.float16)
    with pytest.raises(ValueError, match="inplace:"):
        g.layer_norm(x, inplace=True)
    with pytest.raises(ValueError, match="rstd:"):
        g.layer_norm_backward(x, x, None, OnDeviceVector(0, f32, 2), OnDeviceVector(0, f32, 3))


def test_sizes_past_32_bits_are_refused(monkeypatch):
    """The library takes 32-bit sizes, to which ctypes would cut a larger one without a word."""
    monkeypatch.setattr(g, "_device", lambda: 0)
    bf16, i64, big = torch.bfloat16, torch.int64, (1 << 32) + 2
    x = OnDevice(0, bf16, (2, 8))
    with pytest.raises(ValueError, match="x: sizes below"):
        g.layer_norm(OnDevice(0, bf16, (big, 8)))
    with pytest.raises(ValueError, match="head: sizes below"):
        g.cross_entropy(x, OnDevice(0, bf16, (big, 8)))
    with pytest.raises(ValueError, match="table: sizes below"):
        g.embedding(OnDevice(0, bf16, (2, 1 << 31)), OnDeviceVector(0, i64, 2))
    with pytest.raises(ValueError, match="tokens: sizes below"):
        g.embedding(x, OnDeviceVector(0, i64, big))
    with pytest.raises(ValueError, match="vocab:"):
        g.embedding_backward(x, OnDeviceVector(0, i64, 2), big)


def test_cross_entropy_plan():
    for wave in (68, 76):
        assert g.cross_entropy_plan(4096, 131072, 4096, wave=wave) == (512, False)
        assert g.cross_entropy_plan(300, 8005, 520, wave=wave) == (256, False)
        assert g.cross_entropy_plan(1500, 50001, 2056, wave=wave)[1]  # rows off 128-byte boundaries, large products
        assert not g.cross_entropy_plan(64, 131072, 4104, wave=wave)[1]
        assert g.cross_entropy_plan(4096, 131072, 1024, input_grad=False, wave=wave)[0] == 512  # (its depth is the rows)
        assert g.cross_entropy_plan(1024, 131072, 4096, input_grad=False, wave=wave)[0] == 256
    for bad in ((-1, 8, 8), (8, -1, 8), (8, 8, -1)):
        with pytest.raises(g.GemmError):
            g.cross_entropy_plan(*bad)
    with pytest.raises(g.GemmError):
        g.cross_entropy_plan(8, 8, 8, wave=0)
    assert g.lib().gemm_cross_entropy_plan(8, 8, 8, 76, 0, 1, 1, None, None) == BAD
