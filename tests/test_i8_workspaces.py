"""Workspaces of the integer products by sizes alone (no GPU)."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from sparse_spherical_convolution_gb300 import build
    build.build()
    import sparse_spherical_convolution_gb300 as d
    return d


SHAPES = [(96, 2048, 2048, 1), (5000, 64, 48, 1), (2, 128, 256, 259920), (3, 80, 77, 65341), (1, 24, 40, 5_000_001)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_one_size_for_both_types_of_gradients(lib, shape):
    for f in (lib.disco_matmul_i8_bwd_input_workspace_bytes, lib.disco_matmul_i8_bwd_weight_workspace_bytes):
        assert f(*shape, lib.DISCO_BF16) == f(*shape, lib.DISCO_F16) > 0


@pytest.mark.parametrize("tokens", [1 << 15, 1 << 20, 1 << 24, 1 << 28])
def test_parts_of_long_reductions(lib, tokens):
    """At least a part of 4 bytes to a weight for every 32768 tokens, and no more than twice that and one for each of 152 SMs."""
    cin, cout = 2048, 1280
    n = lib.disco_matmul_i8_bwd_weight_workspace_bytes(tokens, cin, cout, 1) // (4 * cin * cout)
    assert (tokens >> 15 if tokens > 1 << 15 else 0) <= n <= 2 * (tokens >> 15) + 152
