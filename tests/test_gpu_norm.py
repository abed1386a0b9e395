"""disco_rms_norm, disco_rms_norm_bwd and disco_dequant_e4m3 against 64-bit
forms (tests/_train_ops.py, where the bounds are derived): shapes from one
element up, odd pixel counts, channel counts around the kernels' limits, every
type, groups that do not divide C, zero rows, infinities and NaN, in-place
buffers, writes outside the outputs, other streams, 64-bit offsets, gradients
against differences, and refusals."""
import ctypes

import pytest
import torch

from tests._train_ops import TINY, U32, UNIT, assert_close, e4m3_half_step, norm64, norm_bwd64, quant64

pytestmark = pytest.mark.gpu
F32, BF, F16 = torch.float32, torch.bfloat16, torch.float16
EPS = 1e-5


@pytest.fixture(scope="module")
def lib():
    from sparse_spherical_convolution_gb300 import build
    build.build()
    import sparse_spherical_convolution_gb300 as d
    d.disco_device_status(clear=True)
    return d


def _randn(shape, dtype, seed, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype)


class Guarded:
    """A device tensor inside a larger buffer whose rest must keep its bytes."""

    def __init__(self, shape, dtype, fill=None):
        n = 1
        for v in shape:
            n *= v
        size = n * torch.empty((), dtype=dtype).element_size()
        self.pad, self.size = 64, size
        self.buf = torch.full((size + 2 * self.pad,), 0xA5, dtype=torch.uint8, device="cuda")
        self.t = self.buf[self.pad:self.pad + size].view(dtype).view(shape)
        if fill is not None:
            self.t.copy_(fill)

    def check(self, what):
        rest = torch.cat([self.buf[:self.pad], self.buf[self.pad + self.size:]])
        assert bool((rest == 0xA5).all()), f"{what}: bytes beside the output were written"


def _run(lib, x, residual, weight, y=True, q=False, group=0, stream=None):
    B, C, P = x.shape
    G = group if 0 < group < C else C
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    out = {}
    if residual is not None:
        out["h"] = Guarded((B, C, P), x.dtype)
    if y:
        out["y"] = Guarded((B, C, P), x.dtype)
    if q:
        out["q"] = Guarded((B, C, P), torch.float8_e4m3fn)
        out["scale"] = Guarded((B, -(-C // G), P), F32)
    t = {k: v.t for k, v in out.items()}
    lib.disco_rms_norm(dev(x), dev(residual), dev(weight), EPS, t.get("h"), t.get("y"), B, C, P, q=t.get("q"),
                       scale=t.get("scale"), group=group, stream=stream)
    torch.cuda.synchronize()
    for k, g in out.items():
        g.check(k)
    return t


def _check(t, x, residual, weight, group):
    C, dt = x.shape[1], x.dtype
    h, y = norm64(x, residual, weight, EPS)
    rel = (C / 2 + 8) * U32
    if "h" in t:
        # one fp32 sum, one rounding to the type
        assert_close(t["h"], h, (U32 + UNIT[dt] * (1 + U32)) * h.abs() + TINY[dt], "h")
    if "y" in t:
        assert_close(t["y"], y, (rel + UNIT[dt] * (1 + rel)) * y.abs() + TINY[dt], "y")
    if "q" in t:
        scale, v = quant64(y, group)
        assert_close(t["scale"], scale, (rel + 4 * U32) * scale + TINY[F32], "scale")
        slack = 2 * (rel + 4 * U32) * v.abs()
        assert_close(t["q"].float(), v, e4m3_half_step(v.abs() + slack) + slack, "q")


# (B, C, P): one element, one channel, one pixel; rows (P = 1) of odd, ordinary
# and long features; pixel counts below, at and above a vector and a tile, odd
# and even; channel counts around the register-held limits and beyond them
SHAPES = [
    (1, 1, 1), (2, 1, 5), (1, 3, 1), (5, 7, 1), (3, 8, 1), (33, 31, 1), (16, 512, 1), (7, 1000, 1), (3, 2049, 1),
    (2, 8192, 1), (2, 16384, 1), (1, 20011, 1), (2, 40000, 1), (1, 300, 2), (2, 5, 3), (1, 33, 7), (3, 17, 31), (2, 80, 32), (1, 64, 33),
    (1, 4, 64), (2, 48, 255), (1, 256, 256), (1, 100, 1000), (2, 32, 8192), (1, 3, 4099), (1, 129, 513), (1, 512, 264),
    (1, 513, 72), (1, 1024, 40), (1, 1025, 33), (1, 2100, 16), (1, 5000, 9),
]

# more than one tile or row to a thread: tiles past the resident clusters, rows
# past the resident teams; pixel counts 2, 4 and odd modulo 8 with the channels
# of a pixel in one CTA and over a cluster; rows shorter than a vector
LONG = [
    (4, 8, 60000), (4, 8, 60001), (3, 24, 30002), (2, 40, 250), (3, 24, 12), (1, 520, 333), (1, 1100, 58), (2, 300, 1201),
    (5000, 3, 1), (20011, 7, 1), (3000, 257, 1), (2000, 1000, 1), (1300, 2048, 1), (300, 9000, 1), (40, 33000, 1), (1, 40000, 3),
]


@pytest.mark.parametrize("dtype", [F32, BF, F16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_norm_matches_64_bits(lib, shape, dtype):
    B, C, P = shape
    x, r = _randn(shape, dtype, 1), _randn(shape, dtype, 2, 3.0)
    w = _randn((C,), dtype, 3)
    _check(_run(lib, x, r, w), x, r, w, 0)
    _check(_run(lib, x, None, None), x, None, None, 0)
    for group in {0, min(C, 32), max(1, C // 3), 1}:
        _check(_run(lib, x, r, w, y=group == 0, q=True, group=group), x, r, w, group)
    _check(_run(lib, x, None, w, y=True, q=True, group=C + 5), x, None, w, C + 5)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", LONG, ids=lambda s: "x".join(map(str, s)))
def test_norm_of_many_tiles(lib, shape, dtype):
    B, C, P = shape
    x, r, w = _randn(shape, dtype, 31), _randn(shape, dtype, 32, 3.0), _randn((C,), dtype, 33)
    for group in (0, min(C, 32), max(1, C // 3)):
        _check(_run(lib, x, r, w, y=group == 0, q=True, group=group), x, r, w, group)


def _run_bwd(lib, dy, h, weight, dh, dweight=True):
    B, C, P = h.shape
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    dx, dw = Guarded((B, C, P), h.dtype), Guarded((C,), h.dtype) if dweight else None
    ws = None
    if dweight:
        n = lib.disco_rms_norm_bwd_workspace_bytes(B, C, P, lib.dtype_code(h.dtype))
        assert n > 0
        ws = Guarded((n,), torch.uint8)
    lib.disco_rms_norm_bwd(dev(dy), dev(h), dev(weight), dev(dh), EPS, dx.t, dw.t if dweight else None, B, C, P,
                           ws.t if dweight else None)
    torch.cuda.synchronize()
    dx.check("dx")
    if dweight:
        dw.check("dweight")
        ws.check("workspace")
    return dx.t, dw.t if dweight else None


@pytest.mark.parametrize("dtype", [F32, BF, F16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_gradient_matches_64_bits(lib, shape, dtype):
    B, C, P = shape
    dy, h, dh = _randn(shape, dtype, 4), _randn(shape, dtype, 5, 2.0), _randn(shape, dtype, 6)
    w = _randn((C,), dtype, 7)
    for weight, skip, want_dw in ((w, dh, True), (None, None, True), (w, None, False)):
        dx, dw = _run_bwd(lib, dy, h, weight, skip, want_dw)
        rx, S, rw, Sw = norm_bwd64(dy, h, weight, skip, EPS)
        assert_close(dx, rx, (2 * C + 16) * U32 * S + UNIT[dtype] * rx.abs() * 1.01 + TINY[dtype], "dx")
        if want_dw:
            assert_close(dw, rw, (B * P + C / 2 + 8) * U32 * Sw + UNIT[dtype] * rw.abs() * 1.01 + TINY[dtype], "dweight")
            dx2, dw2 = _run_bwd(lib, dy, h, weight, skip, True)
            assert torch.equal(dx, dx2) and torch.equal(dw, dw2)   # fixed order of summation


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", LONG, ids=lambda s: "x".join(map(str, s)))
def test_gradient_of_many_tiles(lib, shape, dtype):
    """The sum over pixels: a thread adds the pixels of its tiles, 16 or 32 lanes
    and then the CTAs join pairwise, so B P terms are off by far less than B P u;
    the bound stays B P u."""
    B, C, P = shape
    dy, h, dh, w = _randn(shape, dtype, 34), _randn(shape, dtype, 35, 2.0), _randn(shape, dtype, 36), _randn((C,), dtype, 37)
    dx, dw = _run_bwd(lib, dy, h, w, dh)
    rx, S, rw, Sw = norm_bwd64(dy, h, w, dh, EPS)
    assert_close(dx, rx, (2 * C + 16) * U32 * S + UNIT[dtype] * rx.abs() * 1.01 + TINY[dtype], "dx")
    assert_close(dw, rw, (B * P + C / 2 + 8) * U32 * Sw + UNIT[dtype] * rw.abs() * 1.01 + TINY[dtype], "dweight")
    # nothing but the tile's own pixels enters: a NaN stays in its pixel and out of other channels' sums of later calls
    h2 = h.clone()
    h2[0, 0, 0] = float("nan")
    dx2, _ = _run_bwd(lib, dy, h2, w, dh)
    clean = torch.ones((B, C, P), dtype=torch.bool)
    clean[0, :, 0] = False
    assert torch.equal(dx2.cpu()[clean], dx.cpu()[clean]) and bool(torch.isnan(dx2[0, :, 0]).all())


@pytest.mark.parametrize("shape", [(2, 6, 1), (1, 40, 12), (3, 9, 35)], ids=lambda s: "x".join(map(str, s)))
def test_gradient_matches_differences(lib, shape):
    """Central differences of the 64-bit loss sum(dy y) + sum(dh h) along random
    directions; their error is O(step^2) = 1e-8 relative, the gradient's as above."""
    B, C, P = shape
    x, r = _randn(shape, F32, 8), _randn(shape, F32, 9)
    dy, dh, w = _randn(shape, F32, 10), _randn(shape, F32, 11), _randn((C,), F32, 12)
    h32 = (x.double() + r.double()).float()
    dx, dw = _run_bwd(lib, dy, h32, w, dh)

    def loss(hh, ww):
        _, y = norm64(hh, None, ww, EPS)
        return float((dy.double() * y).sum() + (dh.double() * hh).sum())

    step = 1e-4
    for seed in range(3):
        v, vw = _randn(shape, torch.float64, 20 + seed), _randn((C,), torch.float64, 30 + seed)
        h64, w64 = h32.double(), w.double()
        diff = (loss(h64 + step * v, w64 + step * vw) - loss(h64 - step * v, w64 - step * vw)) / (2 * step)
        terms = (dx.double().cpu() * v).abs().sum() + (dw.double().cpu() * vw).abs().sum()
        got = float((dx.double().cpu() * v).sum() + (dw.double().cpu() * vw).sum())
        assert abs(got - diff) <= 1e-5 * float(terms), (got, diff)


def test_zero_rows_and_values_outside_the_range(lib):
    """A pixel whose channels are all 0 gives 0; NaN and infinities stay in
    their own pixel; squares past fp32 give 0, as stated."""
    B, C, P = 2, 40, 21
    for dtype in (F32, BF):
        x, w = _randn((B, C, P), dtype, 13), _randn((C,), dtype, 14)
        x[:, :, 3] = 0
        x[0, 5, 7] = float("nan")
        x[1, 6, 8] = float("inf")
        x[0, :, 9] = 1e20
        t = _run(lib, x, None, w, y=True, q=True, group=16)
        y, q, s = t["y"].float().cpu(), t["q"].float().cpu(), t["scale"].cpu()
        assert bool((y[:, :, 3] == 0).all()) and bool((q[:, :, 3] == 0).all())
        assert bool((s[:, :, 3] == torch.tensor(1e-30) / 448).all())
        assert bool(torch.isnan(y[0, :, 7]).all()) and bool(torch.isnan(q[0, :, 7]).all())
        assert bool(torch.isnan(y[1, 6, 8])) and bool((y[1, [c for c in range(C) if c != 6], 8] == 0).all())
        assert bool(torch.isnan(q[1, 6, 8])) and bool((q[1, :6, 8] == 0).all())
        assert bool((y[0, :, 9] == 0).all())
        keep = [p for p in range(P) if p not in (3, 7, 8, 9)]
        part = {"y": t["y"][:, :, keep], "q": t["q"].float()[:, :, keep], "scale": t["scale"][:, :, keep]}
        _check(part, x[:, :, keep], None, w, 16)
        g = _randn((B, C, P), dtype, 15)
        dx, dw = _run_bwd(lib, g, x, w, None)
        rx, S, _, _ = norm_bwd64(g, x, w, None, EPS)
        keep.append(3)
        assert_close(dx[:, :, keep], rx[:, :, keep],
                     (2 * C + 16) * U32 * S[:, :, keep] + UNIT[dtype] * rx[:, :, keep].abs() * 1.01 + TINY[dtype], "dx")
        assert bool(torch.isnan(dx[0, :, 7]).all()) and bool(torch.isnan(dw).any())


def test_tiny_and_huge_groups(lib):
    """Group maxima near the smallest and largest fp32: scales stay positive,
    nothing overflows."""
    C, P = 64, 40
    x = _randn((1, C, P), F32, 16)
    for gain in (1e-37, 1e-25, 1e30):
        w = torch.full((C,), gain)
        t = _run(lib, x, None, w, y=True, q=True, group=32)
        assert bool((t["scale"] > 0).all()) and bool(torch.isfinite(t["scale"]).all())
        assert bool(torch.isfinite(t["q"].float()).all())
        _check(t, x, None, w, 32)


@pytest.mark.parametrize("shape", [(3, 96, 1), (1, 30, 65), (2, 64, 512), (1, 3000, 8)], ids=lambda s: "x".join(map(str, s)))
def test_in_place(lib, shape):
    B, C, P = shape
    x, r, w = _randn(shape, BF, 17).cuda(), _randn(shape, BF, 18).cuda(), _randn((C,), BF, 19).cuda()
    h, y = torch.empty_like(x), torch.empty_like(x)
    lib.disco_rms_norm(x, r, w, EPS, h, y, B, C, P)
    x1, r1 = x.clone(), r.clone()
    lib.disco_rms_norm(x1, r1, w, EPS, r1, x1, B, C, P)      # h over the residual, y over x
    assert torch.equal(r1, h) and torch.equal(x1, y)
    dy, dh = _randn(shape, BF, 20).cuda(), _randn(shape, BF, 21).cuda()
    ws = torch.empty(lib.disco_rms_norm_bwd_workspace_bytes(B, C, P), dtype=torch.uint8, device="cuda")
    dx, dw, dw1 = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    lib.disco_rms_norm_bwd(dy, h, w, dh, EPS, dx, dw, B, C, P, ws)
    for k in range(3):
        bufs = [dy.clone(), h.clone(), dh.clone()]
        lib.disco_rms_norm_bwd(bufs[0], bufs[1], w, bufs[2], EPS, bufs[k], dw1, B, C, P, ws)
        assert torch.equal(bufs[k], dx) and torch.equal(dw1, dw)


@pytest.mark.parametrize("dtype", [F32, BF, F16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (5, 100, 1), (3, 2051, 1), (2, 33, 7), (1, 64, 4096), (3, 20, 1001),
                                   (2, 48, 130), (1, 70, 30004), (2, 129, 5001), (4000, 33, 1)],
                         ids=lambda s: "x".join(map(str, s)))
def test_dequant(lib, shape, dtype):
    B, C, P = shape
    q = _randn(shape, F32, 22, 100.0).clamp(-448, 448).to(torch.float8_e4m3fn)
    for group in (0, 1, 16, 33, C + 1):
        G = group if 0 < group < C else C
        scale = torch.rand((B, -(-C // G), P), generator=torch.Generator().manual_seed(23)) * 1e-2
        out = Guarded(shape, dtype)
        lib.disco_dequant_e4m3(q.cuda(), scale.cuda(), out.t, B, C, P, group)
        torch.cuda.synchronize()
        out.check("x")
        want = (q.float() * scale.repeat_interleave(G, 1)[:, :C]).to(dtype)   # one fp32 product, one rounding
        assert torch.equal(out.t.cpu(), want)


def test_dequant_of_every_code(lib):
    q = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).view(1, 1, 256).cuda()
    one, x = torch.ones((1, 1, 256), device="cuda"), torch.empty((1, 1, 256), device="cuda")
    lib.disco_dequant_e4m3(q, one, x, 1, 1, 256)
    want = q.float()
    assert torch.equal(torch.isnan(x), torch.isnan(want)) and torch.equal(torch.nan_to_num(x), torch.nan_to_num(want))


def test_streams(lib):
    """The calls run on the stream they are given: behind work queued there, and
    two of them at once."""
    shape = (2, 64, 4096)
    x, w = _randn(shape, F32, 24).cuda(), _randn((64,), F32, 25).cuda()
    want = torch.empty_like(x)
    lib.disco_rms_norm(x, None, w, EPS, None, want, *shape)
    ws = torch.empty(lib.disco_rms_norm_bwd_workspace_bytes(*shape, lib.DISCO_F32), dtype=torch.uint8, device="cuda")
    dxw, dww = torch.empty_like(x), torch.empty_like(w)
    lib.disco_rms_norm_bwd(want, x, w, None, EPS, dxw, dww, *shape, ws)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    big = torch.zeros(1 << 26, device="cuda")
    res = []
    for s in streams:
        with torch.cuda.stream(s):
            late, y = torch.empty_like(x), torch.empty_like(x)
            dx, dw, ws2 = torch.empty_like(x), torch.empty_like(w), torch.empty_like(ws)
            for _ in range(4):
                big2 = big + 1                       # keeps the stream busy before x arrives
            late.copy_(x)
        lib.disco_rms_norm(late, None, w, EPS, None, y, *shape, stream=s)
        lib.disco_rms_norm_bwd(y, late, w, None, EPS, dx, dw, *shape, ws2, stream=s.cuda_stream)
        res.append((y, dx, dw, late, ws2, big2))
    torch.cuda.synchronize()
    for y, dx, dw, *_ in res:
        assert torch.equal(y, want) and torch.equal(dx, dxw) and torch.equal(dw, dww)


@pytest.mark.parametrize("shape", [(2, 48, 4096), (40, 1000, 1)], ids=lambda s: "x".join(map(str, s)))
def test_graph_capture(lib, shape):
    """The calls can be captured; a replay sees the inputs of its own time."""
    B, C, P = shape
    x, r, w = _randn(shape, BF, 41).cuda(), _randn(shape, BF, 42).cuda(), _randn((C,), BF, 43).cuda()
    h, y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty(lib.disco_rms_norm_bwd_workspace_bytes(*shape), dtype=torch.uint8, device="cuda")

    def calls():
        lib.disco_rms_norm(x, r, w, EPS, h, y, *shape)
        lib.disco_rms_norm_bwd(y, h, w, r, EPS, dx, dw, *shape, ws)

    calls()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    x.mul_(2)
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (h, y, dx, dw)]
    calls()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (h, y, dx, dw)))
    _check({"h": h, "y": y}, x.cpu(), r.cpu(), w.cpu(), 0)


def test_offsets_past_32_bits(lib):
    """3 channels of 2^30 + 8 pixels: offsets pass 2^31 elements and 2^32 bytes.
    The last and first pixels are compared."""
    C, P = 3, (1 << 30) + 8
    x = torch.full((1, C, P), 0.5, dtype=BF, device="cuda")
    tail = _randn((1, C, 64), BF, 26)
    x[:, :, -64:] = tail.cuda()
    w = _randn((C,), BF, 27)
    y = torch.zeros_like(x)
    lib.disco_rms_norm(x, None, w.cuda(), EPS, None, y, 1, C, P)
    _check({"y": y[:, :, -64:]}, tail, None, w, 0)
    _check({"y": y[:, :, :64]}, torch.full((1, C, 64), 0.5, dtype=BF), None, w, 0)
    dx = torch.zeros_like(x)
    lib.disco_rms_norm_bwd(y, x, w.cuda(), None, EPS, dx, None, 1, C, P)
    yt = y[:, :, -64:].cpu()
    rx, S, _, _ = norm_bwd64(yt, tail, w, None, EPS)
    assert_close(dx[:, :, -64:], rx, (2 * C + 16) * U32 * S + UNIT[BF] * rx.abs() * 1.01 + TINY[BF], "dx")
    del dx, y
    q = torch.zeros((1, C, P), dtype=torch.uint8, device="cuda")
    q[:, :, -1] = 0x38                                # 1.0
    s = torch.full((1, 1, P), 0.25, device="cuda")
    lib.disco_dequant_e4m3(q, s, x, 1, C, P)
    assert bool((x[:, :, -1] == 0.25).all()) and bool((x[:, :, -1000:-1] == 0).all()) and bool((x[:, :, :1000] == 0).all())


def test_refusals(lib):
    B, C, P = 2, 16, 24
    n = (B, C, P)
    x, r, h, y = (torch.zeros(n, dtype=BF, device="cuda") for _ in range(4))
    w, q = torch.zeros(C, dtype=BF, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
    s = torch.zeros((B, 1, P), device="cuda")
    y.fill_(7.0)

    def refused(status, text, fn, *args, **kw):
        with pytest.raises(lib.DiscoError) as e:
            fn(*args, **kw)
        assert e.value.status == status and text in str(e.value), str(e.value)

    norm, bwd = lib.disco_rms_norm, lib.disco_rms_norm_bwd
    refused(-1, "neither y nor q", norm, x, r, w, EPS, h, None, B, C, P)
    refused(-1, "come together", norm, x, r, w, EPS, h, y, B, C, P, q=q)
    refused(-1, "come together", norm, x, r, w, EPS, h, y, B, C, P, scale=s)
    refused(-1, "h without", norm, x, None, w, EPS, h, y, B, C, P)
    refused(-1, "group", norm, x, r, w, EPS, h, y, B, C, P, q=q, scale=s, group=-1)
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        refused(-1, "eps", norm, x, r, w, eps, h, y, B, C, P)
    refused(-1, "elements", norm, x, r, w, EPS, h, y, B, C, P + 1)
    refused(-1, "dtype", norm, x, r.float(), w, EPS, h, y, B, C, P)
    refused(-2, "dtype", norm, x.double(), None, None, EPS, None, x.double(), B, C, P)
    refused(-1, "contiguous", norm, x.transpose(1, 2), None, None, EPS, None, y, B, C, P)
    refused(-1, "CUDA device", norm, x.cpu(), None, w, EPS, None, y, B, C, P)
    refused(-1, "overlaps", norm, x, r, w, EPS, y, y, B, C, P)                    # two outputs in one buffer
    two = torch.zeros(B * C * P + 8, dtype=BF, device="cuda")
    refused(-1, "overlaps", norm, two[:-8], None, w, EPS, None, two[8:], B, C, P)  # in place, shifted
    refused(-1, "overlaps", norm, x, None, w, EPS, None, None, B, C, P, q=x.view(torch.uint8).view(-1)[:B * C * P],
            scale=s)
    refused(-3, "aligned", norm, two[1:1 + B * C * P], None, w, EPS, None, y, B, C, P)
    need = lib.disco_rms_norm_bwd_workspace_bytes(B, C, P)
    small = torch.zeros(need - 4, dtype=torch.uint8, device="cuda")
    refused(-7, "workspace", bwd, x, r, w, None, EPS, y, w.clone(), B, C, P)
    refused(-7, "workspace", bwd, x, r, w, None, EPS, y, w.clone(), B, C, P, small)
    refused(-1, "overlaps", bwd, x, r, w, None, EPS, y, w, B, C, P, torch.zeros(need, dtype=torch.uint8, device="cuda"))
    refused(-1, "dy is None", bwd, None, r, w, None, EPS, y, None, B, C, P)
    refused(-1, "overlaps", lib.disco_dequant_e4m3, x.view(torch.uint8).view(-1)[:B * C * P], s, x, B, C, P)
    refused(-1, "dtype", lib.disco_dequant_e4m3, x, s, y, B, C, P)
    assert lib.disco_rms_norm_bwd_workspace_bytes(0, C, P) == 0
    so, null = lib.load_library(), None
    # through the C ABI: null, empty sizes and host pointers are refused before any launch
    xp, yp = ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(y.data_ptr())
    assert so.disco_rms_norm(null, null, null, EPS, null, yp, null, null, 0, B, C, P, 1, null) == -1
    for b, c, p in ((0, C, P), (B, 0, P), (B, C, 0), (B, C, -1)):
        assert so.disco_rms_norm(xp, null, null, EPS, null, yp, null, null, 0, b, c, p, 1, null) == -1
        assert so.disco_rms_norm_bwd(xp, xp, null, null, EPS, yp, null, b, c, p, 1, null, 0, null) == -1
        assert so.disco_dequant_e4m3(xp, xp, yp, 0, b, c, p, 1, null) == -1
    assert so.disco_rms_norm(xp, null, null, EPS, null, yp, null, null, 0, B, C, P, 9, null) == -2
    host = (ctypes.c_uint16 * (B * C * P + 8))()
    base = (ctypes.addressof(host) + 15) // 16 * 16
    assert so.disco_rms_norm(ctypes.c_void_p(base), null, null, EPS, null, yp, null, null, 0, B, C, P, 1, null) == -1
    assert "device memory" in lib.disco_last_error()
    torch.cuda.synchronize()
    assert bool((y == 7.0).all())
