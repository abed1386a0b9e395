"""Refusals and host-side rules of the 8-bit integer feed-forward that need no GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from sparse_spherical_convolution_gb300 import build
    build.build()
    import sparse_spherical_convolution_gb300 as d
    return d


P = ctypes.c_void_p(256)


def _products(so, args, dtype, ws=None, wn=1 << 40):
    tail = (*args, dtype, ws or P, wn, None)
    return {"fwd": so.disco_matmul_i8(P, P, P, P, P, *tail), "dx": so.disco_matmul_i8_bwd_input(P, P, P, P, *tail),
            "dW": so.disco_matmul_i8_bwd_weight(P, P, P, P, *tail)}


@pytest.mark.parametrize("args", [(0, 8, 8, 1), (1, 0, 8, 1), (1, 8, 0, 1), (1, 8, 8, 0), (-1, 8, 8, 4), (1, 8, 8, -3)])
def test_sizes_are_checked_before_the_device(lib, args):
    so = lib.load_library()
    b, cin, cout, p = args
    for name in ("disco_matmul_i8", "disco_matmul_i8_bwd_input", "disco_matmul_i8_bwd_weight"):
        assert getattr(lib, name + "_workspace_bytes")(*args) == 0
    assert set(_products(so, args, 1).values()) == {-1}
    if min(b, cin, p) < 1:
        assert so.disco_quant_i8(P, P, P, b, cin, p, 1, None) == -1
        assert so.disco_glu(P, P, None, None, None, None, 0, b, cin, p, 1, None) == -1
        assert so.disco_glu_bwd(P, P, P, P, 0, b, cin, p, 1, None) == -1


def test_types_and_pointers_are_checked_before_the_device(lib):
    so = lib.load_library()
    ok = (2, 8, 8, 4)
    assert set(_products(so, ok, 3).values()) == {-2}
    assert set(_products(so, ok, -1).values()) == {-2}
    f32 = _products(so, ok, 0)
    assert f32["dx"] == -2 and f32["dW"] == -2 and "bf16 or fp16" in lib.disco_last_error()
    assert lib.disco_matmul_i8_bwd_input_workspace_bytes(*ok, lib.DISCO_F32) == 0
    assert lib.disco_matmul_i8_workspace_bytes(*ok, lib.DISCO_F32) > 0
    assert so.disco_matmul_i8(P, P, P, None, P, *ok, 1, P, 1 << 40, None) == -1
    assert so.disco_matmul_i8_bwd_input(P, P, None, P, *ok, 1, P, 1 << 40, None) == -1
    assert so.disco_matmul_i8_bwd_weight(P, P, P, None, *ok, 1, P, 1 << 40, None) == -1
    assert so.disco_quant_i8(P, P, P, 2, 8, 4, 7, None) == -2
    assert so.disco_quant_i8(P, None, P, 2, 8, 4, 1, None) == -1
    assert so.disco_quant_i8(P, P, P, 1 << 30, 1 << 20, 1 << 20, 1, None) == -2
    assert so.disco_glu(P, P, None, None, None, None, 2, 2, 8, 4, 1, None) == -2
    assert "activation" in lib.disco_last_error()
    assert so.disco_glu(P, None, None, None, P, P, 0, 2, 8, 4, 1, None) == -1
    assert so.disco_glu(P, P, P, None, None, None, 0, 2, 8, 4, 1, None) == -1
    assert so.disco_glu(P, P, None, None, None, P, 0, 2, 8, 4, 1, None) == -1
    assert so.disco_glu(None, P, None, None, None, None, 0, 2, 8, 4, 1, None) == -1
    assert so.disco_glu(P, P, None, None, None, None, 0, 2, 1 << 30, 4, 1, None) == -2
    assert so.disco_glu_bwd(P, P, None, P, 0, 2, 8, 4, 1, None) == -1
    assert so.disco_glu_bwd(P, P, P, P, -1, 2, 8, 4, 1, None) == -2


def test_limits_of_the_products(lib):
    so = lib.load_library()
    for args in ((1, 8, 8, 1 << 31), (1, 1 << 20, 8, 1 << 21), (1, 1 << 21, 1 << 20, 1)):
        assert set(_products(so, args, 1).values()) == {-2}
        for name in ("disco_matmul_i8", "disco_matmul_i8_bwd_input", "disco_matmul_i8_bwd_weight"):
            assert getattr(lib, name + "_workspace_bytes")(*args) == 0
    assert lib.disco_matmul_i8_workspace_bytes(1, 8, 8, (1 << 31) - 1) > 0


def test_workspace_is_checked_before_the_device(lib):
    so = lib.load_library()
    for args in ((1, 8, 8, 1), (3, 80, 77, 65341), (96, 2048, 2048, 1), (2, 128, 256, 259920)):
        for name, ptrs in (("disco_matmul_i8", 5), ("disco_matmul_i8_bwd_input", 4), ("disco_matmul_i8_bwd_weight", 4)):
            n = getattr(lib, name + "_workspace_bytes")(*args)
            assert n > 0
            assert getattr(so, name)(*[P] * ptrs, *args, 1, P, n - 1, None) == -7
            assert getattr(so, name)(*[P] * ptrs, *args, 1, None, n, None) == -7


def test_binding_rejects_host_tensors(lib):
    import torch
    x, q = torch.zeros((2, 8, 4)), torch.zeros((2, 8, 4), dtype=torch.int8)
    s, W = torch.zeros((2, 4)), torch.zeros((8, 8), dtype=torch.int8)
    for call in (lambda: lib.disco_quant_i8(x, q, s, 2, 8, 4),
                 lambda: lib.disco_matmul_i8(q, s, W, s, x, 2, 8, 8, 4),
                 lambda: lib.disco_matmul_i8_bwd_input(x, W, s, x, 2, 8, 8, 4),
                 lambda: lib.disco_matmul_i8_bwd_weight(x, q, s, x, 2, 8, 8, 4),
                 lambda: lib.disco_glu(x, x, lib.DISCO_SILU, 2, 4, 4),
                 lambda: lib.disco_glu_bwd(x, q, s, x, lib.DISCO_SILU, 2, 4, 4)):
        with pytest.raises(lib.DiscoError) as e:
            call()
        assert e.value.status == -1 and "CUDA device" in str(e.value)
