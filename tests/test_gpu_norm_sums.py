"""dweight of disco_rms_norm_bwd at shapes with many tiles or rows to a thread,
within a bound that a lost or doubled tile would exceed.

Bound.  The workspace holds one row of partial sums for each CTA or cluster, so
its size tells their number R.  With N = B P pixels, a thread adds at most
N / R of them and up to 8 of an uneven last tile (it holds one pixel of 8 at
most, but that is left out), then come at most 5 additions over lanes, 16 over
the teams of a CTA, R / 32 + 1 over the rows of partial sums and 5 over the lanes
there: fewer than N / R + R / 32 + 48 roundings of 2^-24 on a term's way.  A term
dy h r is off by C / 2 + 8 of them (the sum of squares by C, its root by half of
that) and 3 for its products.  Terms of either sign: all relative to the sum of
their magnitudes.  Then one rounding to the type.

That the bound is narrow enough is tested too: a vector of zeros exceeds it in most
channels, and in fp32 the 64-bit sums without 64 pixels (one row of features where
P = 1), at the start, the middle and the end, exceed it in some.  The 16-bit types'
own rounding of a sum can hide so few pixels."""
import pytest
import torch

from tests._train_ops import TINY, U32, UNIT, assert_close, norm_bwd64
from tests.test_gpu_norm import EPS, LONG, _randn, _run_bwd

F32, BF, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def lib():
    from sparse_spherical_convolution_gb300 import build
    build.build()
    import sparse_spherical_convolution_gb300 as d
    return d


def _inputs(shape, dtype):
    return _randn(shape, dtype, 51), _randn(shape, dtype, 52, 2.0), _randn((shape[1],), dtype, 53)


def _sums(lib, shape, dtype, dy, h, w):
    """dweight in 64 bits and its bound."""
    B, C, P = shape
    R = lib.disco_rms_norm_bwd_workspace_bytes(B, C, P, lib.dtype_code(dtype)) // (4 * C)
    assert R >= 1
    _, _, rw, Sw = norm_bwd64(dy, h, w, None, EPS)
    return rw, (B * P / R + R / 32 + 48 + C / 2 + 11) * U32 * Sw + UNIT[dtype] * rw.abs() * 1.01 + TINY[dtype]


CASES = [(s, dt) for s in LONG for dt in (F32, BF, F16)]
IDS = ["x".join(map(str, s)) + "-" + str(dt)[6:] for s, dt in CASES]


@pytest.mark.gpu
@pytest.mark.parametrize("shape,dtype", CASES, ids=IDS)
def test_dweight_of_many_tiles(lib, shape, dtype):
    dy, h, w = _inputs(shape, dtype)
    _, dw = _run_bwd(lib, dy, h, w, None)
    rw, bound = _sums(lib, shape, dtype, dy, h, w)
    assert_close(dw, rw, bound, "dweight")


@pytest.mark.parametrize("shape,dtype", CASES, ids=IDS)
def test_the_bound_shows_a_lost_tile(lib, shape, dtype):
    B, C, P = shape
    dy, h, w = _inputs(shape, dtype)
    rw, bound = _sums(lib, shape, dtype, dy, h, w)
    assert float((rw.abs() > bound).double().mean()) > 0.8       # zeros
    if dtype is not F32:
        return
    n = min(64, P)
    for b, p in ((0, 0), (B // 2, (P - n) // 2), (B - 1, P - n)):
        _, _, lost, _ = norm_bwd64(dy[b:b + 1, :, p:p + n], h[b:b + 1, :, p:p + n], w, None, EPS)
        assert bool((lost.abs() > bound).any()), (b, p, float((lost.abs() / bound).max()))
