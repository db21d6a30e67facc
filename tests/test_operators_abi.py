"""Argument checks of the operators around the products (no GPU needed: refusals come before any device use)."""
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
