"""The 8-bit integer feed-forward against plain 64-bit forms (bounds: tests/_i8_ops.py)."""
import math
import zlib

import pytest
import torch

from tests import _i8_ops as r

pytestmark = pytest.mark.gpu

F32, BF, HF = torch.float32, torch.bfloat16, torch.float16
ALL, HALF = [F32, BF, HF], [BF, HF]
ids = lambda t: str(t)[6:] if isinstance(t, torch.dtype) else str(t)  # noqa: E731


@pytest.fixture(scope="module")
def lib():
    from sparse_spherical_convolution_gb300 import build
    build.build()
    import sparse_spherical_convolution_gb300 as d
    return d


def _gen(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def _randn(g, *shape):
    return torch.randn(shape, generator=g)


# tokens: one, rows with and without whole words, grids, odd grids, few and many channels
TOKENS = [(1, 1, 1), (1, 512, 1), (3, 17, 1), (33, 100, 1), (130, 256, 1), (5, 1365, 1), (2, 4097, 1), (2, 9000, 1), (1, 16384, 1),
          (1, 1, 2), (2, 5, 7), (1, 3, 64), (3, 16, 128), (2, 80, 181), (1, 64, 33 * 65), (2, 130, 1000), (1, 700, 96), (1, 2050, 40), (4, 9, 4099),
          (1, 5000, 24), (1, 520, 33), (1, 900, 301), (1, 1700, 77), (2, 40, 1001), (1, 7500, 16), (1, 1200, 200), (2, 6, 1030)]


def _x(shape, dtype, seed=0):
    g = _gen("x", shape, seed)
    x = _randn(g, *shape) * torch.exp(_randn(g, 1, shape[1], 1))
    x = x.to(dtype)
    # values on and next to borders: halves of the largest, and its neighbours
    a = x.abs().amax(1, keepdim=True)
    pick = torch.rand(shape, generator=g)
    x = torch.where(pick < 0.05, a / 2, x)
    x = torch.where(pick > 0.95, -a / 2, x)
    return x.to(dtype)


@pytest.mark.parametrize("dtype", ALL, ids=ids)
@pytest.mark.parametrize("shape", TOKENS, ids=ids)
def test_quant_is_the_definition(lib, shape, dtype):
    B, C, P = shape
    x = _x(shape, dtype)
    q, q_ok = r.guarded(shape, torch.int8)
    s, s_ok = r.guarded((B, P), F32)
    lib.disco_quant_i8(x.cuda(), q, s, B, C, P)
    want, scale = r.quant64(x)
    assert torch.equal(q.cpu().double(), want), (q.cpu().double() != want).sum()
    r.assert_close(s, scale, scale * 2 * r.U32, "scale")
    q_ok(), s_ok()


@pytest.mark.parametrize("dtype", ALL, ids=ids)
@pytest.mark.parametrize("P", [1, 8, 5])
def test_quant_of_special_tokens(lib, P, dtype):
    """Zeros, the largest and smallest magnitudes, infinities and NaN; a token's
    neighbours keep their values."""
    big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).tiny
    rows = [[0.0, 0.0, -0.0], [big, -big, big / 2], [tiny, -tiny, 0.0], [1.0, float("inf"), 2.0], [1.0, float("nan"), 2.0],
            [float("-inf"), float("nan"), 0.0], [3.0, -1.5, 0.75]]
    B, C = len(rows), 3
    x = torch.tensor(rows).to(dtype)[:, :, None].repeat(1, 1, P).contiguous()
    if P > 1:
        x[:, :, 1] = torch.tensor([1.0, -2.0, 0.25]).to(dtype)
    q, s = torch.empty((B, C, P), dtype=torch.int8, device="cuda"), torch.empty((B, P), device="cuda")
    lib.disco_quant_i8(x.cuda(), q, s, B, C, P)
    q, s = q.cpu(), s.cpu()
    fin = torch.isfinite(x.double()).all(1)
    want, scale = r.quant64(torch.where(fin[:, None], x.double(), torch.zeros(())))
    assert torch.equal(torch.where(fin[:, None], q.double(), torch.zeros((), dtype=torch.float64)), want)
    r.assert_close(s[fin], scale[fin], scale[fin] * 2 * r.U32, "scale")
    assert not torch.isfinite(s[~fin]).any()
    back = q.float() * s[:, None]
    assert torch.isnan(back.permute(0, 2, 1)[~fin]).all()


# products: one token, few, more than a tile, odd channel counts; grids whole, odd, with more than one sample
SHAPES = [(1, 1, 1, 1), (1, 512, 2048, 1), (3, 17, 5, 1), (8, 256, 64, 1), (16, 1024, 33, 1), (33, 100, 77, 1), (130, 64, 257, 1), (200, 130, 48, 1),
          (17, 2048, 96, 1), (129, 1030, 300, 1), (2, 48, 5000, 1), (5, 33, 4900, 1), (16, 100, 4871, 1), (1, 4100, 4865, 1),
          (1, 3, 5, 2), (2, 5, 3, 7), (1, 16, 16, 64), (3, 64, 48, 128), (2, 80, 77, 181), (1, 64, 48, 33 * 65), (2, 130, 140, 1000), (4, 9, 300, 272),
          (1, 300, 9, 16), (1, 520, 136, 304)]


def _operands(shape, dtype, seed=0):
    B, Cin, Cout, P = shape
    g = _gen("mm", shape, seed)
    q = torch.randint(-127, 128, (B, Cin, P), generator=g, dtype=torch.int8)
    W = torch.randint(-127, 128, (Cout, Cin), generator=g, dtype=torch.int8)
    scale = torch.exp(_randn(g, B, P) - 4)
    wscale = torch.exp(_randn(g, Cout) - 6)
    return q, scale, W, wscale, (0.01 * _randn(g, B, Cout, P)).to(dtype if dtype != F32 else BF)


def _ws(n):
    return torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dtype", ALL, ids=ids)
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_matmul(lib, shape, dtype):
    B, Cin, Cout, P = shape
    q, scale, W, wscale, _ = _operands(shape, dtype)
    y, ok = r.guarded((B, Cout, P), dtype)
    ws = _ws(lib.disco_matmul_i8_workspace_bytes(*shape, lib.dtype_code(dtype)))
    lib.disco_matmul_i8(q.cuda(), scale.cuda(), W.cuda(), wscale.cuda(), y, *shape, ws)
    want, S = r.matmul64(q, scale, W, wscale)
    r.assert_close(y, want, r.matmul_bound(want, S, scale, wscale, Cin, dtype), "y")
    ok()
    assert lib.disco_device_status() == 0


@pytest.mark.parametrize("dtype", HALF, ids=ids)
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_matmul_gradients(lib, shape, dtype):
    B, Cin, Cout, P = shape
    q, scale, W, wscale, dy = _operands(shape, dtype)
    code = lib.dtype_code(dtype)
    dx, dx_ok = r.guarded((B, Cin, P), dtype)
    dW, dW_ok = r.guarded((Cout, Cin), dtype)
    lib.disco_matmul_i8_bwd_input(dy.cuda(), W.cuda(), wscale.cuda(), dx, *shape,
                                  _ws(lib.disco_matmul_i8_bwd_input_workspace_bytes(*shape, code)))
    lib.disco_matmul_i8_bwd_weight(dy.cuda(), q.cuda(), scale.cuda(), dW, *shape,
                                   _ws(lib.disco_matmul_i8_bwd_weight_workspace_bytes(*shape, code)))
    want, S, D = r.bwd_input64(dy, W, wscale)
    r.assert_close(dx, want, r.grad_bound(want, S, D, Cout, dtype), "dx")
    want, S, D = r.bwd_weight64(dy, q, scale)
    r.assert_close(dW, want, r.grad_bound(want, S, D, B * P, dtype), "dW")
    dx_ok(), dW_ok()
    assert lib.disco_device_status() == 0


@pytest.mark.parametrize("dtype", HALF, ids=ids)
@pytest.mark.parametrize("shape", [(2, 128, 256, 16400), (2, 128, 256, 16401), (6000, 512, 384, 1), (6001, 515, 391, 1), (1, 1024, 520, 4112),
                                   (3, 80, 77, 9999), (1, 4096, 1000, 1), (40, 8200, 136, 1), (20000, 512, 256, 1), (2, 515, 300, 9001),
                                   (20001, 300, 520, 1)], ids=ids)
def test_many_steps_and_tiles(lib, shape, dtype):
    """Reductions of many steps, split or not, over many tiles: the rings of shared
    memory go round often.  Five runs give the same bits."""
    B, Cin, Cout, P = shape
    q, scale, W, wscale, dy = [t.cuda() for t in _operands(shape, dtype)]
    code = lib.dtype_code(dtype)
    y, dx = torch.empty((B, Cout, P), dtype=dtype, device="cuda"), torch.empty((B, Cin, P), dtype=dtype, device="cuda")
    dW = torch.empty((Cout, Cin), dtype=dtype, device="cuda")
    ws = _ws(max(f(*shape, code) for f in (lib.disco_matmul_i8_workspace_bytes, lib.disco_matmul_i8_bwd_input_workspace_bytes,
                                           lib.disco_matmul_i8_bwd_weight_workspace_bytes)))
    first = None
    for _ in range(5):
        for t in (y, dx, dW):
            t.fill_(float("nan"))
        lib.disco_matmul_i8(q, scale, W, wscale, y, *shape, ws)
        lib.disco_matmul_i8_bwd_input(dy, W, wscale, dx, *shape, ws)
        lib.disco_matmul_i8_bwd_weight(dy, q, scale, dW, *shape, ws)
        if first is None:
            first = [t.clone() for t in (y, dx, dW)]
        assert all(torch.equal(a, b) for a, b in zip(first, (y, dx, dW)))
    assert lib.disco_device_status() == 0
    cpu = lambda *ts: [t.cpu() for t in ts]  # noqa: E731
    want, S = r.matmul64(q, scale, W, wscale)
    r.assert_close(y, *cpu(want, r.matmul_bound(want, S, scale, wscale, Cin, dtype)), "y")
    want, S, D = r.bwd_input64(dy, W, wscale)
    r.assert_close(dx, *cpu(want, r.grad_bound(want, S, D, Cout, dtype)), "dx")
    want, S, D = r.bwd_weight64(dy, q, scale)
    r.assert_close(dW, *cpu(want, r.grad_bound(want, S, D, B * P, dtype)), "dW")


@pytest.mark.parametrize("shape", [(20000, 512, 256, 1), (20001, 100, 250, 1), (2, 128, 256, 16400), (2, 128, 256, 16401), (1, 64, 700, 7000)], ids=ids)
def test_large_products_in_32_bits(lib, shape):
    B, Cin, Cout, P = shape
    q, scale, W, wscale, _ = [t.cuda() for t in _operands(shape, F32)]
    y, ok = r.guarded((B, Cout, P), F32)
    lib.disco_matmul_i8(q, scale, W, wscale, y, *shape, _ws(lib.disco_matmul_i8_workspace_bytes(*shape, lib.DISCO_F32)))
    want, S = r.matmul64(q, scale, W, wscale)
    r.assert_close(y, want.cpu(), r.matmul_bound(want, S, scale, wscale, Cin, F32).cpu(), "y")
    ok()


@pytest.mark.parametrize("P", [1, 37, 64])
def test_extreme_integers_and_scales(lib, P):
    """-128 and 127 everywhere (the sum is exact for Cin <= 1024), and scales that
    are infinite or NaN stay with their token or channel."""
    B, Cin, Cout = (70, 1024, 130) if P == 1 else (2, 1024, 130)
    q, W = torch.full((B, Cin, P), -128, dtype=torch.int8), torch.full((Cout, Cin), 127, dtype=torch.int8)
    W[1::2] = -128
    scale, wscale = torch.full((B, P), 2.0 ** -10), torch.full((Cout,), 2.0 ** -12)
    y = torch.empty((B, Cout, P), device="cuda")
    ws = _ws(lib.disco_matmul_i8_workspace_bytes(B, Cin, Cout, P, lib.DISCO_F32))
    lib.disco_matmul_i8(q.cuda(), scale.cuda(), W.cuda(), wscale.cuda(), y, B, Cin, Cout, P, ws)
    want, _ = r.matmul64(q, scale, W, wscale)
    assert torch.equal(y.cpu().double(), want)
    scale[1, 0], wscale[5] = float("nan"), float("inf")
    lib.disco_matmul_i8(q.cuda(), scale.cuda(), W.cuda(), wscale.cuda(), y, B, Cin, Cout, P, ws)
    got = y.cpu().double()
    assert torch.isnan(got[1, :, 0]).all() and torch.isinf(got[0, 5]).all()
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[1, :, 0] = False
    keep[:, 5] = False
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("dtype", HALF, ids=ids)
def test_gradients_keep_what_is_infinite_apart(lib, dtype):
    """An infinity or a NaN of dy reaches the outputs of its token or channel alone."""
    for shape in ((70, 40, 24, 1), (2, 40, 24, 100), (2, 40, 24, 96)):
        B, Cin, Cout, P = shape
        q, scale, W, wscale, dy = _operands(shape, dtype)
        code = lib.dtype_code(dtype)
        clean = dy.clone()
        dy[1, 3, 0] = float("nan")
        dx, dW = torch.empty((B, Cin, P), dtype=dtype, device="cuda"), torch.empty((Cout, Cin), dtype=dtype, device="cuda")
        lib.disco_matmul_i8_bwd_input(dy.cuda(), W.cuda(), wscale.cuda(), dx, *shape,
                                      _ws(lib.disco_matmul_i8_bwd_input_workspace_bytes(*shape, code)))
        lib.disco_matmul_i8_bwd_weight(dy.cuda(), q.cuda(), scale.cuda(), dW, *shape,
                                       _ws(lib.disco_matmul_i8_bwd_weight_workspace_bytes(*shape, code)))
        want, S, D = r.bwd_input64(clean, W, wscale)
        want[1, :, 0] = float("nan")
        r.assert_close(dx, want, r.grad_bound(want, S, D, Cout, dtype), "dx")
        want, S, D = r.bwd_weight64(clean, q, scale)
        want[3] = float("nan")
        r.assert_close(dW, want, r.grad_bound(want, S, D, B * P, dtype), "dW")


def test_gradients_are_those_of_differences(lib):
    """The loss sum(dy y) is linear in the activation and in the weight: its change
    for a change of one of them is dx and dW."""
    for shape in ((9, 32, 16, 1), (2, 24, 40, 48)):
        B, Cin, Cout, P = shape
        q, scale, W, wscale, dy = _operands(shape, BF)
        dx, dW = torch.empty((B, Cin, P), dtype=BF, device="cuda"), torch.empty((Cout, Cin), dtype=BF, device="cuda")
        lib.disco_matmul_i8_bwd_input(dy.cuda(), W.cuda(), wscale.cuda(), dx, *shape, _ws(lib.disco_matmul_i8_bwd_input_workspace_bytes(*shape)))
        lib.disco_matmul_i8_bwd_weight(dy.cuda(), q.cuda(), scale.cuda(), dW, *shape, _ws(lib.disco_matmul_i8_bwd_weight_workspace_bytes(*shape)))

        def loss(q_, W_):
            y, S = r.matmul64(q_, scale, W_, wscale)
            return (dy.double() * y).sum().item(), (dy.double().abs() * S).sum().item()
        (base, _) = loss(q, W)
        q2 = q.clone().double()
        q2[1, 2] += 3
        got = (dx[1, 2].cpu().double() * 3 * scale[1].double()).sum().item()
        want, S, D = r.bwd_input64(dy, W, wscale)
        tol = (r.grad_bound(want, S, D, Cout, BF)[1, 2] * 3 * scale[1].double()).sum().item()
        assert abs(loss(q2, W)[0] - base - got) <= tol
        W2 = W.clone().double()
        W2[3, 4] -= 5
        got = dW[3, 4].item() * -5 * wscale[3].item()
        want, S, D = r.bwd_weight64(dy, q, scale)
        tol = r.grad_bound(want, S, D, B * P, BF)[3, 4].item() * 5 * wscale[3].item()
        assert abs(loss(q, W2)[0] - base - got) <= tol


# ------------------------------------------------------------------ gated activation

GLU = [(1, 1, 1), (1, 512, 1), (3, 17, 1), (33, 100, 1), (130, 256, 1), (5, 1365, 1), (2, 4097, 1), (1, 12000, 1), (1, 1, 2), (2, 5, 7), (3, 16, 128), (2, 80, 181),
       (2, 130, 1000), (1, 700, 96), (1, 3000, 24), (1, 300, 33), (1, 600, 200), (1, 1100, 40), (2, 6, 1032), (1, 4000, 16),
       (3, 20, 1001), (1, 9, 4099), (2, 33, 2145), (1, 1000, 137), (2, 7, 65), (1, 64, 66)]


@pytest.mark.parametrize("dtype", ALL, ids=ids)
@pytest.mark.parametrize("shape", GLU, ids=ids)
@pytest.mark.parametrize("outs", ["y", "q", "yq", "yx", "qx", "yqx"])
def test_glu(lib, shape, dtype, outs):
    B, C, P = shape
    act = (B + C + P) % 2
    x = (1.5 * _randn(_gen("glu", shape), B, 2 * C, P)).to(dtype)
    y, y_ok = r.guarded((B, C, P), dtype)
    q, q_ok = r.guarded((B, C, P), torch.int8)
    s, s_ok = r.guarded((B, P), F32)
    xq, xq_ok = r.guarded((B, 2 * C, P), torch.int8)
    xs, xs_ok = r.guarded((B, P), F32)
    has = lambda k, *t: t if k in outs else (None,) * len(t)  # noqa: E731
    (oy,), (oq, os), (oxq, oxs) = has("y", y), has("q", q, s), has("x", xq, xs)
    lib.disco_glu(x.cuda(), oy, act, B, C, P, q=oq, scale=os, xq=oxq, xscale=oxs)
    want, e = r.glu64(x, act)
    if "y" in outs:
        r.assert_close(y, want, want.abs() * (e + r.UNIT[dtype]) + r.TINY[dtype], "y")
    if "q" in outs:
        a = want.abs().amax(1).clamp_min(r.FLOOR)
        ea = e.amax(1)
        r.assert_close(s, a / 127, a / 127 * (ea + 4 * r.U32), "scale")
        r.assert_close(q, 127 * want / a[:, None], (0.5 + 254 * (ea + 4 * r.U32))[:, None].expand_as(want), "q")
    if "x" in outs:
        wq, ws = r.quant64(x)
        assert torch.equal(xq.cpu().double(), wq)
        r.assert_close(xs, ws, ws * 2 * r.U32, "xscale")
    y_ok(), q_ok(), s_ok(), xq_ok(), xs_ok()


@pytest.mark.parametrize("act", [0, 1], ids=["silu", "gelu"])
@pytest.mark.parametrize("dtype", ALL, ids=ids)
@pytest.mark.parametrize("shape", GLU, ids=ids)
def test_glu_bwd(lib, shape, dtype, act):
    B, C, P = shape
    g = _gen("glub", shape)
    xq = torch.randint(-127, 128, (B, 2 * C, P), generator=g, dtype=torch.int8)
    xs = (0.01 + 0.05 * torch.rand((B, P), generator=g))
    dy = _randn(g, B, C, P).to(dtype)
    dx, ok = r.guarded((B, 2 * C, P), dtype)
    lib.disco_glu_bwd(dy.cuda(), xq.cuda(), xs.cuda(), dx, act, B, C, P)
    want, bound = r.glu_bwd64(dy, xq, xs, act, dtype)
    r.assert_close(dx, want, bound, "dx")
    ok()


@pytest.mark.parametrize("act", [0, 1], ids=["silu", "gelu"])
def test_glu_gradient_is_that_of_differences(lib, act):
    """Central differences of the 64-bit formula, step 1e-4: off by h^2/6 |act'''| |dy v| < 1e-8 of it."""
    B, C, P = 2, 12, 16
    g = _gen("diff", act)
    xq = torch.randint(-127, 128, (B, 2 * C, P), generator=g, dtype=torch.int8)
    xs, dy = torch.full((B, P), 0.03), _randn(g, B, C, P)
    dx = torch.empty((B, 2 * C, P), device="cuda")
    lib.disco_glu_bwd(dy.cuda(), xq.cuda(), xs.cuda(), dx, act, B, C, P)
    x, h = xq.double() * xs.double()[:, None], 1e-4
    _, bound = r.glu_bwd64(dy, xq, xs, act, F32)
    for half in (0, 1):
        step = torch.zeros_like(x)
        step[:, half * C:(half + 1) * C] = h
        num = (r.glu64(x + step, act)[0] - r.glu64(x - step, act)[0]) * dy.double() / (2 * h)
        at = slice(half * C, (half + 1) * C)
        scale = (dy.double() * x[:, C:]).abs() + dy.double().abs()
        r.assert_close(dx[:, at], num, bound[:, at] + 1e-7 * scale, "dx")


@pytest.mark.parametrize("dtype", ALL, ids=ids)
@pytest.mark.parametrize("P", [1, 8, 5])
def test_glu_special_values(lib, dtype, P):
    """Large gates of both signs saturate, zeros stay zeros, a NaN stays with its token."""
    C = 4
    x = torch.zeros((2, 2 * C, P))
    x[0, :, 0] = torch.tensor([80.0, -80.0, 0.0, 1.0, 2.0, 2.0, 5.0, 0.0])
    x[1, 0, P - 1] = float("nan")
    x = x.to(dtype).cuda()
    y, q = torch.empty((2, C, P), dtype=dtype, device="cuda"), torch.empty((2, C, P), dtype=torch.int8, device="cuda")
    s = torch.empty((2, P), device="cuda")
    for act in (0, 1):
        lib.disco_glu(x, y, act, 2, C, P, q=q, scale=s)
        yc = y.double().cpu()
        assert yc[0, 0, 0] == 160 and abs(yc[0, 1, 0]) < 1e-30 and yc[0, 2, 0] == 0 and yc[0, 3, 0] == 0
        assert q[0, :, 0].tolist() == [127, 0, 0, 0]
        assert torch.isnan(yc[1, 0, P - 1]) and torch.isnan(s[1, P - 1])
        if P > 1:
            assert bool((yc[:, :, 1:P - 1] == 0).all()) and bool((s[:, 1:P - 1] < 1e-30).all())


@pytest.mark.parametrize("dtype", ALL, ids=ids)
def test_masked_pixels_and_extreme_tokens_beside_ordinary_ones(lib, dtype):
    """Pixels of zeros, of the largest and of the smallest magnitudes in one tile with ordinary ones."""
    B, C, P = 2, 24, 136
    x = _x((B, C, P), dtype, 7)
    x[:, :, 3::7] = 0
    x[0, :, 5] *= torch.finfo(dtype).max / 1e3 / x[0, :, 5].abs().max().clamp_min(1) if dtype != HF else 8
    x[1, :, 9] = (x[1, :, 9].float() * 1e-25).to(dtype)
    q, s = torch.empty((B, C, P), dtype=torch.int8, device="cuda"), torch.empty((B, P), device="cuda")
    for pixels in (P, P - 3):
        v = x[:, :, :pixels].contiguous()
        qv, sv = q.view(-1)[:v.numel()].view(v.shape), s.view(-1)[:B * pixels].view(B, pixels)
        lib.disco_quant_i8(v.cuda(), qv, sv, B, C, pixels)
        want, scale = r.quant64(v)
        assert torch.equal(qv.cpu().double(), want)
        r.assert_close(sv, scale, scale * 2 * r.U32, "scale")


# ------------------------------------------------------------------ calls

def test_refusals(lib):
    B, Cin, Cout, P = 2, 16, 32, 48
    q = torch.zeros((B, Cin, P), dtype=torch.int8, device="cuda")
    s, W = torch.zeros((B, P), device="cuda"), torch.zeros((Cout, Cin), dtype=torch.int8, device="cuda")
    sw, y = torch.zeros(Cout, device="cuda"), torch.zeros((B, Cout, P), dtype=BF, device="cuda")
    ws = _ws(1 << 24)

    def status(call):
        with pytest.raises(lib.DiscoError) as e:
            call()
        return e.value.status
    mm = lambda **k: lib.disco_matmul_i8(*[k.get(n, v) for n, v in (("q", q), ("s", s), ("W", W), ("sw", sw), ("y", y))],  # noqa: E731
                                         B, Cin, Cout, P, k.get("ws", ws))
    mm()
    assert status(lambda: mm(ws=None)) == -7
    assert status(lambda: mm(q=q.float())) == -1                                       # type
    assert status(lambda: mm(W=W.t())) == -1                                           # strides
    assert status(lambda: mm(q=q[:1])) == -1                                           # size
    off = torch.zeros(B * Cout * P + 1, dtype=BF, device="cuda")[1:]
    assert status(lambda: mm(y=off)) == -3                                             # alignment
    both = torch.zeros(B * Cout * P * 2, dtype=torch.uint8, device="cuda")
    assert status(lambda: mm(q=both[:B * Cin * P].view(torch.int8), y=both.view(BF))) == -1  # overlap
    assert status(lambda: mm(ws=y.view(-1).view(torch.uint8))) == -1
    dy = torch.zeros((B, Cout, P), device="cuda")
    dx = torch.zeros((B, Cin, P), device="cuda")
    assert status(lambda: lib.disco_matmul_i8_bwd_input(dy, W, sw, dx, B, Cin, Cout, P, ws)) == -2
    assert status(lambda: lib.disco_quant_i8(dx, q, None, B, Cin, P)) == -1
    assert status(lambda: lib.disco_quant_i8(dx, dx.view(torch.int8).view(-1)[:q.numel()], s, B, Cin, P)) == -1
    x = torch.zeros((B, 2 * Cin, P), dtype=BF, device="cuda")
    assert status(lambda: lib.disco_glu(x, None, 0, B, Cin, P)) == -1
    assert status(lambda: lib.disco_glu(x, x.view(-1)[:B * Cin * P], 0, B, Cin, P)) == -1
    assert status(lambda: lib.disco_glu(x, torch.empty_like(x[:, :Cin]).contiguous(), 7, B, Cin, P)) == -2
    torch.cuda.synchronize()


def _block(lib, B, C, F, P, dtype, t, ws):
    """norm output n -> n in 8 bits -> gates and values -> 8 bits -> C channels, and all gradients from the 8-bit activations."""
    lib.disco_quant_i8(t["n"], t["nq"], t["ns"], B, C, P)
    lib.disco_matmul_i8(t["nq"], t["ns"], t["W1"], t["s1"], t["u"], B, C, 2 * F, P, ws)
    lib.disco_glu(t["u"], None, lib.DISCO_SILU, B, F, P, q=t["gq"], scale=t["gs"], xq=t["uq"], xscale=t["us"])
    lib.disco_matmul_i8(t["gq"], t["gs"], t["W2"], t["s2"], t["y"], B, F, C, P, ws)
    lib.disco_matmul_i8_bwd_weight(t["dy"], t["gq"], t["gs"], t["dW2"], B, F, C, P, ws)
    lib.disco_matmul_i8_bwd_input(t["dy"], t["W2"], t["s2"], t["dg"], B, F, C, P, ws)
    lib.disco_glu_bwd(t["dg"], t["uq"], t["us"], t["du"], lib.DISCO_SILU, B, F, P)
    lib.disco_matmul_i8_bwd_weight(t["du"], t["nq"], t["ns"], t["dW1"], B, C, 2 * F, P, ws)
    lib.disco_matmul_i8_bwd_input(t["du"], t["W1"], t["s1"], t["dn"], B, C, 2 * F, P, ws)


def _block_tensors(lib, B, C, F, P, dtype, seed=0):
    g = _gen("block", B, C, F, P, seed)
    e = lambda *s, dt=dtype: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    i8 = torch.int8
    t = {"n": _randn(g, B, C, P).to(dtype).cuda(), "dy": (0.1 * _randn(g, B, C, P)).to(dtype).cuda(),
         "nq": e(B, C, P, dt=i8), "ns": e(B, P, dt=F32), "u": e(B, 2 * F, P), "gq": e(B, F, P, dt=i8), "gs": e(B, P, dt=F32),
         "uq": e(B, 2 * F, P, dt=i8), "us": e(B, P, dt=F32), "y": e(B, C, P), "dg": e(B, F, P), "du": e(B, 2 * F, P), "dn": e(B, C, P),
         "dW1": e(2 * F, C), "dW2": e(C, F), "W1": e(2 * F, C, dt=i8), "s1": e(2 * F, dt=F32), "W2": e(C, F, dt=i8), "s2": e(C, dt=F32)}
    for W, s, o, i in (("W1", "s1", 2 * F, C), ("W2", "s2", C, F)):
        lib.disco_quant_i8((_randn(g, o, i) / math.sqrt(i)).cuda(), t[W], t[s], o, i, 1)
    code = lib.dtype_code(dtype)
    n = max(f(B, a, b, P, code) for a, b in ((C, 2 * F), (F, C)) for f in (
        lib.disco_matmul_i8_workspace_bytes, lib.disco_matmul_i8_bwd_input_workspace_bytes, lib.disco_matmul_i8_bwd_weight_workspace_bytes))
    return t, _ws(n)


@pytest.mark.parametrize("dtype", HALF, ids=ids)
@pytest.mark.parametrize("shape", [(40, 96, 160, 1), (2, 48, 72, 33 * 5), (2, 64, 96, 256)], ids=ids)
def test_feed_forward_block(lib, shape, dtype):
    """Each step of the block against the 64-bit form of that step's own inputs."""
    B, C, F, P = shape
    t, ws = _block_tensors(lib, B, C, F, P, dtype)
    _block(lib, B, C, F, P, dtype, t, ws)
    c = {k: v.cpu() for k, v in t.items()}
    assert torch.equal(c["nq"].double(), r.quant64(c["n"])[0])
    assert torch.equal(c["uq"].double(), r.quant64(c["u"])[0])
    for q, s, W, sw, y, K in (("nq", "ns", "W1", "s1", "u", C), ("gq", "gs", "W2", "s2", "y", F)):
        want, S = r.matmul64(c[q], c[s], c[W], c[sw])
        r.assert_close(c[y], want, r.matmul_bound(want, S, c[s], c[sw], K, dtype), y)
    for dy, q, s, dW in (("dy", "gq", "gs", "dW2"), ("du", "nq", "ns", "dW1")):
        want, S, D = r.bwd_weight64(c[dy], c[q], c[s])
        r.assert_close(c[dW], want, r.grad_bound(want, S, D, B * P, dtype), dW)
    for dy, W, s, dx, K in (("dy", "W2", "s2", "dg", C), ("du", "W1", "s1", "dn", 2 * F)):
        want, S, D = r.bwd_input64(c[dy], c[W], c[s])
        r.assert_close(c[dx], want, r.grad_bound(want, S, D, K, dtype), dx)
    want, bound = r.glu_bwd64(c["dg"], c["uq"], c["us"], 0, dtype)
    r.assert_close(c["du"], want, bound, "du")


@pytest.mark.parametrize("shape", [(40, 96, 160, 1), (1, 64, 80, 1), (2, 64, 96, 256), (2, 48, 72, 165)], ids=ids)
def test_streams_graphs_and_repeats_give_the_same(lib, shape):
    """A captured and replayed block, one on another stream, and two at once on two
    streams with workspaces of their own give bit for bit the first run's outputs."""
    B, C, F, P = shape
    outs = ("nq", "gq", "uq", "y", "dW1", "dW2", "dn")
    t, ws = _block_tensors(lib, B, C, F, P, BF)
    _block(lib, B, C, F, P, BF, t, ws)
    torch.cuda.synchronize()
    want = {k: t[k].clone() for k in outs}

    def check(t):
        torch.cuda.synchronize()
        for k in outs:
            assert torch.equal(t[k], want[k]), k
            t[k].zero_()
    check(t)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    t2, ws2 = _block_tensors(lib, B, C, F, P, BF)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        _block(lib, B, C, F, P, BF, t, ws)
    with torch.cuda.stream(other):
        _block(lib, B, C, F, P, BF, t2, ws2)
    check(t), check(t2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _block(lib, B, C, F, P, BF, t, ws)
    ws.fill_(255)
    for _ in range(3):
        graph.replay()
        check(t)
    assert lib.disco_device_status() == 0


def test_offsets_past_32_bits(lib):
    """More than 2^31 elements in one sample: values at both ends."""
    B, C, P = 1, 3, 800_000_000
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty((B, C, P), dtype=BF, device="cuda").normal_(generator=g)
    q, s = torch.empty((B, C, P), dtype=torch.int8, device="cuda"), torch.empty((B, P), device="cuda")
    lib.disco_quant_i8(x, q, s, B, C, P)
    ends = [slice(0, 4096), slice(P // 2 - 2048, P // 2 + 2048), slice(P - 4096, P)]
    for at in ends:
        want, scale = r.quant64(x[:, :, at].cpu())
        assert torch.equal(q[:, :, at].cpu().double(), want)
    del x
    W = torch.randint(-127, 128, (4, C), generator=_gen("W"), dtype=torch.int8)
    sw = torch.rand(4, generator=_gen("s")) * 0.01
    y = torch.empty((B, 4, P), dtype=BF, device="cuda")
    ws = _ws(lib.disco_matmul_i8_workspace_bytes(B, C, 4, P))
    lib.disco_matmul_i8(q, s, W.cuda(), sw.cuda(), y, B, C, 4, P, ws)
    for at in ends:
        sc = s[:, at].cpu()
        want, S = r.matmul64(q[:, :, at].cpu(), sc, W, sw)
        r.assert_close(y[:, :, at], want, r.matmul_bound(want, S, sc, sw, C, BF), "y")
    dx = torch.empty((B, C, P), dtype=BF, device="cuda")
    lib.disco_matmul_i8_bwd_input(y, W.cuda(), sw.cuda(), dx, B, C, 4, P, _ws(lib.disco_matmul_i8_bwd_input_workspace_bytes(B, C, 4, P)))
    for at in ends:
        want, S, D = r.bwd_input64(y[:, :, at].cpu(), W, sw)
        r.assert_close(dx[:, :, at], want, r.grad_bound(want, S, D, 4, BF), "dx")
    # all but the ends' tokens count nothing, so the sum over tokens is the ends'
    y[:, :, 4096:P - 4096] = 0
    dW = torch.empty((4, C), dtype=BF, device="cuda")
    lib.disco_matmul_i8_bwd_weight(y, q, s, dW, B, C, 4, P, _ws(lib.disco_matmul_i8_bwd_weight_workspace_bytes(B, C, 4, P)))
    keep = lambda t: torch.cat([t[..., :4096], t[..., P - 4096:]], -1).cpu()  # noqa: E731
    want, S, D = r.bwd_weight64(keep(y), keep(q), keep(s))
    r.assert_close(dW, want, r.grad_bound(want, S, D, 8192, BF), "dW")
    assert lib.disco_device_status() == 0


@pytest.mark.parametrize("shape", [(3, 64, 40, 1), (70, 1024, 130, 1), (300, 96, 130, 1), (2, 64, 130, 64), (2, 1024, 24, 37)], ids=ids)
def test_scales_whose_product_leaves_fp32(lib, shape):
    """scale * wscale past both ends of fp32 where y is inside.  y takes three
    roundings of 2^-24 (the exact sum's conversion among them) and a subnormal half step."""
    B, Cin, Cout, P = shape
    g = _gen("products", shape)
    q = torch.randint(-127, 128, (B, Cin, P), generator=g, dtype=torch.int8)
    W = torch.randint(-127, 128, (Cout, Cin), generator=g, dtype=torch.int8)
    q[0] = 0
    scale, wscale = torch.full((B, P), 1e-25), torch.full((Cout,), 1e-17)
    scale[0], wscale[1] = 1e25, 1e25
    y = torch.empty((B, Cout, P), device="cuda")
    lib.disco_matmul_i8(q.cuda(), scale.cuda(), W.cuda(), wscale.cuda(), y, B, Cin, Cout, P,
                        _ws(lib.disco_matmul_i8_workspace_bytes(B, Cin, Cout, P, lib.DISCO_F32)))
    want, _ = r.matmul64(q, scale, W, wscale)
    assert (y[0].cpu() == 0).all()
    r.assert_close(y, want, 3 * 2.0 ** -24 * want.abs() + 2.0 ** -150, "y")


def test_as_many_rows_as_fit_the_argument(lib):
    """2^31 - 1 rows of one value: both ends."""
    B = 2 ** 31 - 1
    x = torch.full((B,), 3.0, dtype=BF, device="cuda")
    x[-3:] = torch.tensor([-5.0, 0.0, 7.0])
    q, s = torch.zeros(B, dtype=torch.int8, device="cuda"), torch.zeros(B, device="cuda")
    lib.disco_quant_i8(x, q, s, B, 1, 1)
    assert q[-5:].tolist() == [127, 127, -127, 0, 127] and q[:3].tolist() == [127] * 3
    want, scale = r.quant64(torch.tensor([3.0, 3.0, -5.0, 0.0, 7.0])[:, None, None])
    r.assert_close(s[-5:], scale[:, 0], 2.0 ** -24 * scale[:, 0], "scale")
    assert lib.disco_device_status() == 0


def test_host_threads_at_once(lib):
    """Four threads, each with its own tensors, workspace and stream, give what one gives."""
    import threading
    shapes = [(40, 96, 160, 1), (2, 64, 96, 256), (2, 48, 72, 165), (1, 64, 80, 1)]
    outs = ("nq", "gq", "uq", "y", "dW1", "dW2", "dn")
    runs, errors = [], []
    for B, C, F, P in shapes:
        t, ws = _block_tensors(lib, B, C, F, P, BF)
        _block(lib, B, C, F, P, BF, t, ws)
        torch.cuda.synchronize()
        want = {k: t[k].clone() for k in outs}
        for k in outs:
            t[k].zero_()
        runs.append(((B, C, F, P, BF, t, ws), want, torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(args, stream):
        try:
            with torch.cuda.stream(stream):
                for _ in range(20):
                    _block(lib, *args)
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(args, stream)) for args, _, stream in runs]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not errors
    for args, want, _ in runs:
        for k in outs:
            assert torch.equal(args[5][k], want[k]), (args[:4], k)
    assert lib.disco_device_status() == 0


@pytest.mark.parametrize("shape", [(16, 2048, 70, 1), (16, 2049, 70, 1), (4, 8192, 40, 1), (4, 8193, 40, 1), (1, 32768, 40, 1), (1, 32769, 40, 1),
                                   (12, 6929, 3079, 1)], ids=ids)
def test_few_rows_up_to_the_kernels_limit(lib, shape):
    """Both sides of where rows are too long for the kernel of a few rows."""
    B, Cin, Cout, P = shape
    q, scale, W, wscale, _ = _operands(shape, F32)
    y = torch.empty((B, Cout, P), device="cuda")
    lib.disco_matmul_i8(q.cuda(), scale.cuda(), W.cuda(), wscale.cuda(), y, B, Cin, Cout, P,
                        _ws(lib.disco_matmul_i8_workspace_bytes(B, Cin, Cout, P, lib.DISCO_F32)))
    want, S = r.matmul64(q, scale, W, wscale)
    r.assert_close(y, want, r.matmul_bound(want, S, scale, wscale, Cin, F32), "y")
    assert lib.disco_device_status() == 0
