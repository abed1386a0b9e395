"""Refusals and host-side rules of the training operators that need no GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from sparse_spherical_convolution_gb300 import build
    build.build()
    import sparse_spherical_convolution_gb300 as d
    return d


def test_norm_arguments_are_checked_before_the_device(lib):
    so, p = lib.load_library(), ctypes.c_void_p(256)
    for b, c, n in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (-1, 4, 4)):
        assert so.disco_rms_norm(p, None, None, 1e-5, None, p, None, None, 0, b, c, n, 1, None) == -1
        assert so.disco_rms_norm_bwd(p, p, None, None, 1e-5, p, None, b, c, n, 1, None, 0, None) == -1
        assert so.disco_dequant_e4m3(p, p, p, 0, b, c, n, 1, None) == -1
        assert lib.disco_rms_norm_bwd_workspace_bytes(b, c, n) == 0
    assert so.disco_rms_norm(p, None, None, 1e-5, None, p, None, None, 0, 1, 1, 1, 3, None) == -2
    assert so.disco_rms_norm(None, None, None, 1e-5, None, p, None, None, 0, 1, 1, 1, 1, None) == -1
    assert so.disco_rms_norm(p, None, None, 0.0, None, p, None, None, 0, 1, 1, 1, 1, None) == -1
    assert "eps" in lib.disco_last_error()
    assert so.disco_rms_norm(p, None, None, 1e-5, None, None, None, None, 0, 1, 1, 1, 1, None) == -1
    assert so.disco_rms_norm(p, p, None, 1e-5, None, p, None, None, -2, 1, 1, 1, 1, None) == -1
    assert so.disco_rms_norm_bwd(p, p, None, None, 1e-5, p, p, 1, 8, 8, 1, None, 0, None) == -7
    assert so.disco_rms_norm(p, None, None, 1e-5, None, p, None, None, 0, 1 << 30, 1 << 20, 1 << 20, 1, None) == -2


def test_workspace_covers_the_partial_sums(lib):
    for b, c, p in ((1, 1, 1), (3, 80, 65341), (16384, 2048, 1), (2, 128, 259920)):
        n = lib.disco_rms_norm_bwd_workspace_bytes(b, c, p)
        assert n >= 4 * c and n % (4 * c) == 0
        assert n <= 4 * c * b * p


def test_grad_plan_host_rules(lib):
    so, c = lib.load_library(), lib.disco_grads()
    assert so.disco_grad_plan(None, 0, ctypes.byref(c)) == 0 and c.count == 0 and c.numel == 0
    assert lib.disco_grad_workspace_bytes(c) > 0
    t = (lib.disco_grad_tensor * 2)()                  # two tensors without elements: any pointers
    assert so.disco_grad_plan(t, 2, ctypes.byref(c)) == 0 and c.count == 2 and c.has_out == 1
    t[0].n, t[0].grad = 4, 256
    t[0].dtype = 5
    assert so.disco_grad_plan(t, 2, ctypes.byref(c)) == -2
    t[0].dtype, t[0].grad = lib.DISCO_F32, 258
    assert so.disco_grad_plan(t, 2, ctypes.byref(c)) == -3
    t[0].grad = None
    assert so.disco_grad_plan(t, 2, ctypes.byref(c)) == -1
    assert c.count == 0                                 # a refused plan is empty
    assert so.disco_grad_plan(t, -1, ctypes.byref(c)) == -1
    assert so.disco_grad_norm(None, 1.0, None, None, 0, None) == -1
    assert so.disco_grad_norm(ctypes.byref(c), 0.0, None, None, 0, None) == -1


def test_binding_rejects_host_tensors(lib):
    import torch
    x = torch.zeros((1, 2, 3))
    with pytest.raises(lib.DiscoError) as e:
        lib.disco_rms_norm(x, None, None, 1e-5, None, x, 1, 2, 3)
    assert e.value.status == -1
    with pytest.raises(lib.DiscoError):
        lib.GradPlan([x])
    assert lib.dtype_code(torch.float16) == lib.DISCO_F16
    with pytest.raises(lib.DiscoError):
        lib.dtype_code(torch.float64)
