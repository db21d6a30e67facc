"""Argument checks of the operators around the products (no GPU needed: refusals come before any device use)."""
import importlib.util
import os

import pytest
import torch

import dense_tensor_core_persistent_gb300 as g
from dense_tensor_core_persistent_gb300 import build as gbuild

BAD, SHAPE, ALIGN = g.GEMM_ERR_INVALID_ARG, g.GEMM_ERR_UNSUPPORTED_SHAPE, g.GEMM_ERR_MISALIGNED


@pytest.fixture(scope="module", autouse=True)
def built():
    gbuild.build()


def norm(x=16, r=0, w=16, s=0, y=16, scales=0, rstd=0, rows=2, cols=32, eps=1e-5, fmt=0, strides=None):
    return g.lib().gemm_rms_norm(x, r, w, s, y, scales, rstd, rows, cols, eps, fmt, 0, strides)


def norm_backward(dy=16, s=16, w=16, rstd=16, ds=0, dx=16, dw=16, rows=2, cols=32, strides=None):
    return g.lib().gemm_rms_norm_backward(dy, s, w, rstd, ds, dx, dw, rows, cols, 0, strides)


def test_rms_norm_refusals():
    assert norm(rows=0, x=0, y=0) == g.GEMM_OK and norm(cols=0, x=0, y=0) == g.GEMM_OK
    assert norm(rows=-1) == BAD and norm(cols=-1) == BAD
    assert norm(eps=-1.0) == BAD and norm(eps=float("nan")) == BAD
    assert norm(fmt=3) == BAD and norm(fmt=-1) == BAD
    assert norm(x=0) == BAD and norm(y=0) == BAD
    assert norm(fmt=g.GEMM_NORM_E4M3) == BAD  # no scales
    assert norm(r=16, s=0) == BAD  # the sum has nowhere to go
    assert norm(cols=32761) == SHAPE
    assert norm(fmt=g.GEMM_NORM_NVFP4, scales=16, cols=24) == SHAPE
    assert norm(fmt=g.GEMM_NORM_NVFP4, scales=16, x=18) == ALIGN
    assert norm(x=17) == ALIGN and norm(y=17) == ALIGN and norm(rstd=18) == ALIGN
    assert norm(fmt=g.GEMM_NORM_E4M3, scales=18) == ALIGN
    assert norm(strides=g.gemm_norm_strides_t(31, 0, 0, 0)) == BAD
    assert norm(fmt=g.GEMM_NORM_NVFP4, scales=16, strides=g.gemm_norm_strides_t(0, 0, 0, 48)) == SHAPE
    assert norm(fmt=g.GEMM_NORM_NVFP4, scales=16, strides=g.gemm_norm_strides_t(33, 0, 0, 0)) == ALIGN


def test_rms_norm_backward_refusals():
    assert norm_backward(cols=0, dy=0) == g.GEMM_OK
    assert norm_backward(rows=0, dy=0, s=0, rstd=0, dx=0, dw=0) == g.GEMM_OK
    assert norm_backward(rows=-1) == BAD and norm_backward(cols=-3) == BAD
    assert norm_backward(dy=0) == BAD and norm_backward(s=0) == BAD and norm_backward(rstd=0) == BAD
    assert norm_backward(dx=0) == BAD
    assert norm_backward(cols=32761) == SHAPE
    assert norm_backward(dx=17) == ALIGN and norm_backward(dw=18) == ALIGN
    assert norm_backward(strides=g.gemm_norm_backward_strides_t(0, 0, 8, 0)) == BAD


def test_binding_refuses_tensors_that_are_not_what_it_takes():
    x = torch.zeros(2, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        g.rms_norm(x)  # not on a GPU
    with pytest.raises(ValueError):
        g.rms_norm(x, out="int8")


def test_no_device_is_reported():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert norm() == g.GEMM_ERR_NO_DEVICE
    assert norm_backward() == g.GEMM_ERR_NO_DEVICE


def logprobs(l=16, kind=0, tokens=16, lp=16, ent=16, lse=16, top=0, tl=16, ti=16, rows=2, vocab=32, ld=0, scale=1.0):
    return g.lib().gemm_token_logprobs(l, kind, tokens, lp, ent, lse, top, tl, ti, rows, vocab, ld, scale, 0)


def logprobs_backward(l=16, kind=0, tokens=16, lse=16, ent=16, dlp=16, dh=16, dl=16, rows=2, vocab=32, ld=0, ldd=0,
                      scale=1.0):
    return g.lib().gemm_token_logprobs_backward(l, kind, tokens, lse, ent, dlp, dh, dl, rows, vocab, ld, ldd, scale, 0)


def test_token_logprobs_refusals():
    assert logprobs(rows=0, l=0) == g.GEMM_OK
    assert logprobs(rows=-1) == BAD and logprobs(vocab=-1) == BAD and logprobs(vocab=0) == BAD
    assert logprobs(kind=2) == BAD and logprobs(top=-1) == BAD and logprobs(top=33) == SHAPE
    assert logprobs(top=8, vocab=7) == BAD
    assert logprobs(top=3, tl=0) == BAD and logprobs(top=3, ti=0) == BAD
    assert logprobs(l=0) == BAD and logprobs(ent=0) == BAD and logprobs(lse=0) == BAD and logprobs(tokens=0) == BAD
    assert logprobs(ld=31) == BAD and logprobs(ld=-1) == BAD
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert logprobs(scale=scale) == BAD
    assert logprobs(l=17) == ALIGN and logprobs(kind=1, l=18) == ALIGN and logprobs(tokens=20) == ALIGN
    assert logprobs(lse=18) == ALIGN
    assert logprobs(vocab=(1 << 30) + 1) == SHAPE


def test_token_logprobs_backward_refusals():
    assert logprobs_backward(rows=0, l=0) == g.GEMM_OK
    assert logprobs_backward(rows=-1) == BAD and logprobs_backward(vocab=0) == BAD and logprobs_backward(kind=-1) == BAD
    assert logprobs_backward(dlp=0) == BAD and logprobs_backward(tokens=0) == BAD  # one without the other
    assert logprobs_backward(ent=0) == BAD and logprobs_backward(lse=0) == BAD and logprobs_backward(dl=0) == BAD
    assert logprobs_backward(ld=8) == BAD and logprobs_backward(ldd=8) == BAD
    assert logprobs_backward(scale=0.0) == BAD
    assert logprobs_backward(dl=17) == ALIGN and logprobs_backward(dlp=18) == ALIGN


def glu(x=16, wg=16, wu=16, h=16, pre=0, M=2, N=8, K=8, act=0, strides=None):
    return g.lib().gemm_glu_bf16(x, wg, wu, h, pre, M, N, K, act, 0, strides)


def glu8(x=16, xs=16, wg=16, gs=16, wu=16, us=16, h=16, M=2, N=8, K=16, act=0, strides=None):
    return g.lib().gemm_glu_e4m3(x, xs, wg, gs, wu, us, h, M, N, K, act, 0, strides)


def glu_backward(dh=16, x=16, wg=16, wu=16, pre=16, dx=16, dwg=16, dwu=16, M=2, N=8, K=8, act=0, strides=None):
    return g.lib().gemm_glu_bf16_backward(dh, x, wg, wu, pre, dx, dwg, dwu, M, N, K, act, 0, strides)


def test_glu_refusals():
    assert glu(M=0, x=0, h=0) == g.GEMM_OK and glu(N=0, h=0) == g.GEMM_OK
    assert glu(M=-1) == BAD and glu(N=-8) == BAD and glu(K=-8) == BAD and glu(act=3) == BAD and glu(act=-1) == BAD
    assert glu(x=0) == BAD and glu(wg=0) == BAD and glu(wu=0) == BAD and glu(h=0) == BAD
    assert glu(K=12) == SHAPE and glu(N=12) == SHAPE
    assert glu(x=24) == ALIGN and glu(h=8) == ALIGN and glu(pre=8) == ALIGN
    assert glu(strides=g.gemm_glu_strides_t(4, 0, 0, 0)) == BAD
    assert glu(strides=g.gemm_glu_strides_t(12, 0, 0, 0)) == SHAPE
    assert glu(strides=g.gemm_glu_strides_t(0, 12, 0, 0)) == SHAPE


def test_glu_e4m3_refusals():
    assert glu8(M=0, x=0, h=0) == g.GEMM_OK
    assert glu8(M=-1) == BAD and glu8(act=9) == BAD and glu8(xs=0) == BAD and glu8(gs=0) == BAD and glu8(us=0) == BAD
    assert glu8(K=24) == SHAPE and glu8(N=4) == SHAPE and glu8(strides=g.gemm_glu_strides_t(24, 0, 0, 0)) == SHAPE
    assert glu8(x=24) == ALIGN and glu8(xs=18) == ALIGN and glu8(us=17) == ALIGN


def test_glu_backward_refusals():
    assert glu_backward(dx=0, dwg=0, dwu=0) == g.GEMM_OK  # nothing asked for
    assert glu_backward(M=0, dwg=0, dwu=0) == g.GEMM_OK
    assert glu_backward(dwg=0) == BAD and glu_backward(dwu=0) == BAD  # one without the other
    assert glu_backward(dh=0) == BAD and glu_backward(pre=0) == BAD and glu_backward(wg=0) == BAD and glu_backward(x=0) == BAD
    assert glu_backward(M=-1) == BAD and glu_backward(act=7) == BAD
    assert glu_backward(K=4) == SHAPE and glu_backward(N=20) == SHAPE
    assert glu_backward(strides=g.gemm_glu_strides_t(0, 0, 12, 0)) == SHAPE
    assert glu_backward(strides=g.gemm_glu_strides_t(0, 0, 0, 4)) == BAD
    assert glu_backward(dwg=8) == ALIGN and glu_backward(pre=8) == ALIGN


def test_glu_plan():
    assert g.glu_plan(1, 28672, 8192)[0] == 0 and g.glu_plan(128, 28672, 8192)[0] == 0
    assert g.glu_plan(129, 28672, 8192)[0] == 256  # one row of tiles: no gain from taller ones
    assert g.glu_plan(4096, 14336, 4096) == (512, 512)
    assert g.glu_plan(4000, 14336, 1024)[0] == 256  # a shallow sum
    assert g.glu_plan(300, 1368, 520) == (256, 256)
    for bad in ((-1, 8, 8, 76), (8, -8, 8, 76), (8, 8, -8, 76), (8, 8, 8, 0)):
        with pytest.raises(g.GemmError):
            g.glu_plan(*bad)


def test_example_quantises_a_row_of_zeros():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward.py")
    spec = importlib.util.spec_from_file_location("feed_forward", path)
    ff = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ff)
    w = torch.randn(3, 32, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    w[1] = 0.0
    codes, scale = ff.to_e4m3_rows(w)
    assert scale[1] == 0 and torch.all(codes[1].float() == 0)
    back = codes.float() * scale[:, None]
    assert torch.all((back - w.float()).abs() <= 2.0 ** -4 * w.float().abs() + 2.0 ** -10 * scale[:, None])
