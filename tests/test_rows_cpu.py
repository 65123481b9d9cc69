"""CPU tests of the operators on rows: the C ABI refuses bad arguments before any CUDA call,
and the binding refuses host tensors."""
import ctypes
import math

import pytest
import torch

from submanifold_sparse_convolution_hash_gb300 import binding


@pytest.fixture(scope="module")
def libsc():
    from submanifold_sparse_convolution_hash_gb300 import build
    build.build()
    return binding.lib()


def norm(L, rows=4, channels=64, eps=1e-6, dtype=1, out=1, w=256, scale=None):
    return L.sc_add_norm_fwd(None, None, None, None, scale, w, rows, channels, eps, dtype, out, None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=7), 1), (dict(dtype=3, out=3), 1), (dict(out=2), 1), (dict(rows=-1), 1), (dict(rows=1 << 31), 1),
    (dict(channels=0), 5), (dict(channels=12), 5), (dict(channels=16392), 5), (dict(eps=-1.0), 1),
    (dict(eps=math.nan), 1), (dict(eps=math.inf), 1), (dict(w=None), 1), (dict(scale=256), 1), (dict(), 1),
    (dict(out=3), 1), (dict(rows=0), 0), (dict(rows=0, w=None, out=3), 0),
])
def test_norm_refuses_before_any_device_call(libsc, change, status):
    assert norm(libsc, **change) == status


def norm_bwd(L, rows=4, channels=64, eps=1e-6, dtype=1):
    return L.sc_add_norm_bwd(None, None, None, None, None, None, rows, channels, eps, dtype, None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), 1), (dict(rows=-1), 1), (dict(channels=20), 5), (dict(eps=-1.0), 1), (dict(), 1), (dict(rows=0), 0),
])
def test_norm_gradients_refuse_before_any_device_call(libsc, change, status):
    assert norm_bwd(libsc, **change) == status


def linear(L, rows=4, c_in=64, c_out=64, act=0, kind=1, dtype=1, sx=None):
    return L.sc_linear_fwd(None, None, sx, None, None, None, None, None, rows, c_in, c_out, act, kind, dtype, None)


@pytest.mark.parametrize("change,status", [
    (dict(kind=0), 5), (dict(dtype=0), 5), (dict(kind=0, dtype=0), 5), (dict(kind=2), 1), (dict(dtype=3), 1),
    (dict(kind=9), 1), (dict(rows=-1), 1), (dict(rows=1 << 31), 1), (dict(c_in=0), 5), (dict(c_in=12), 5),
    (dict(c_in=65544), 5), (dict(c_out=4), 5), (dict(c_out=65544), 5), (dict(kind=3, c_in=24), 5), (dict(act=4), 1),
    (dict(act=-1), 1), (dict(sx=256), 1), (dict(), 1), (dict(kind=3), 1), (dict(rows=0), 0),
])
def test_linear_refuses_before_any_device_call(libsc, change, status):
    assert linear(libsc, **change) == status


def linear_bwd(L, rows=4, c_in=64, c_out=64, act=0, dtype=1):
    gin = (ctypes.c_int64 * 2)(0, 64)
    return L.sc_linear_bwd(None, None, None, None, gin, None, None, rows, c_in, c_out, act, dtype, None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=0), 5), (dict(dtype=3), 1), (dict(rows=-1), 1), (dict(c_in=4), 5), (dict(c_out=20), 5),
    (dict(act=17), 1), (dict(), 1), (dict(rows=0), 0),
])
def test_linear_gradients_refuse_before_any_device_call(libsc, change, status):
    assert linear_bwd(libsc, **change) == status


def test_clip_refuses_before_any_device_call(libsc):
    assert libsc.sc_grad_clip(None, -1, 1.0, None, None) == 1
    assert libsc.sc_grad_clip(None, 1, 1.0, None, None) == 1
    assert libsc.sc_grad_clip(None, 0, -1.0, None, None) == 1
    assert libsc.sc_grad_clip(None, 0, math.nan, None, None) == 1
    assert libsc.sc_grad_clip(None, 0, 1.0, None, None) == 1  # nowhere for the norm


def test_binding_refuses_host_tensors():
    x = torch.zeros((4, 64), dtype=torch.float16)
    w = torch.ones(64)
    W = torch.zeros((64, 32), dtype=torch.float16)
    for call in (lambda: binding.sc_add_norm_fwd(x, w), lambda: binding.sc_add_norm_bwd(x, x, w),
                 lambda: binding.sc_linear_fwd(x, W), lambda: binding.sc_linear_bwd(x, x, W),
                 lambda: binding.sc_grad_clip([x], 1.0)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="a tensor for each"):
        binding.GradList([x], out=[])
