"""disco_grad_norm, disco_grad_clip and disco_grad_norm_clip against 64-bit
sums: no tensors, empty and one-element tensors, views at odd offsets, lists
longer than one launch takes, mixed types, in place, values near the ends of
fp32's range, infinities and NaN, streams, graphs, and refusals.

Bound of the norm: squares are positive, a thread adds at most 64 of them in
fp32 at these sizes (relative error 64 * 2^-24 of the sum, half of that of its
root), the rest is in 64 bits and one rounding.  An output adds the rounding
of the factor (3 operations), of the product and of the output's type."""
import ctypes
import math

import pytest
import torch

from tests._train_ops import TINY, U32, UNIT

pytestmark = pytest.mark.gpu
F32, BF, F16 = torch.float32, torch.bfloat16, torch.float16
NORM_TOL = 34 * U32


@pytest.fixture(scope="module")
def lib():
    from sparse_spherical_convolution_gb300 import build
    build.build()
    import sparse_spherical_convolution_gb300 as d
    d.disco_device_status(clear=True)
    return d


def _norm64(grads):
    return math.sqrt(math.fsum(float((g.double() ** 2).sum()) for g in grads))


def _call(lib, grads, outs, max_norm, scale=1.0):
    plan = lib.GradPlan(grads, outs)
    norm = torch.full((1,), -1.0, device="cuda")
    ws = torch.full((lib.disco_grad_workspace_bytes(plan.c),), 0xFF, dtype=torch.uint8, device="cuda")
    lib.disco_grad_norm_clip(plan.c, max_norm, norm, ws, grad_scale=scale)
    torch.cuda.synchronize()
    return float(norm)


def _check_out(out, g, factor):
    want = g.double() * factor
    tol = (NORM_TOL + 5 * U32 + UNIT[out.dtype] * 1.01) * want.abs() + TINY[out.dtype] * 1.01
    assert bool(((out.double() - want).abs() <= tol).all())


def _grads(sizes, dtypes, seed, level=1e-2):
    gen = torch.Generator().manual_seed(seed)
    return [(level * torch.randn(n, generator=gen)).to(dt).cuda() for n, dt in zip(sizes, dtypes)]


LISTS = {
    "one": ([1], [F32]),
    "odd": ([1, 3, 4097, 8191, 12289], [F32, BF, F16, BF, F32]),
    "empty among them": ([0, 17, 0, 4096, 0], [BF] * 5),
    "large": ([500_003, 4096 * 7], [BF, F16]),
    "many": ([1 + (37 * i) % 300 for i in range(700)], [(F32, BF, F16)[i % 3] for i in range(700)]),
    "at the table's end": ([40] * 256, [F32] * 256),
}


@pytest.mark.parametrize("name", LISTS)
@pytest.mark.parametrize("mode", ["f32 out", "same type", "in place"])
def test_norm_and_clip(lib, name, mode):
    sizes, dtypes = LISTS[name]
    grads = _grads(sizes, dtypes, 1)
    keep = [g.clone() for g in grads]
    want = _norm64(grads)
    for max_norm, scale in ((0.37 * want, 1.0), (0.2 * want, 0.25), (2 * want, 1.0), (2 * want, 0.5), (math.inf, 1.0), (0.0, 1.0)):
        grads = [g.clone() for g in keep]
        outs = grads if mode == "in place" else [torch.full_like(g, 9.0, dtype=F32 if mode == "f32 out" else g.dtype) for g in grads]
        got = _call(lib, grads, outs, max_norm, scale)
        assert abs(got - scale * want) <= (NORM_TOL + U32) * scale * want
        factor = scale if scale * want <= max_norm else scale * max_norm / (scale * want)
        for o, g in zip(outs, keep):
            _check_out(o, g, factor)
        if mode != "in place":
            assert all(torch.equal(a, b) for a, b in zip(grads, keep))
        elif factor == 1.0:
            assert all(torch.equal(a, b) for a, b in zip(grads, keep))


@pytest.mark.parametrize("shift", [0, 1, 2, 3, 5, 7])
@pytest.mark.parametrize("dtype", [F32, BF, F16], ids=["f32", "bf16", "f16"])
def test_views_at_any_offset(lib, shift, dtype):
    """Gradients and outs packed back to back from any element: every byte
    outside them stays."""
    sizes = [5, 1, 64, 4095, 8200, 3]
    total = sum(sizes)
    src = (1e-2 * torch.randn(total + 32, generator=torch.Generator().manual_seed(2))).to(dtype).cuda()
    for odt, oshift in ((F32, 0), (F32, 3), (dtype, shift), (dtype, (shift + 1) % 8)):
        dst = torch.full((total + 32,), 5.0, dtype=odt, device="cuda")
        grads = list(src[shift:shift + total].split(sizes))
        outs = list(dst[oshift:oshift + total].split(sizes))
        want = _norm64(grads)
        got = _call(lib, grads, outs, want / 3)
        assert abs(got - want) <= (NORM_TOL + U32) * want
        _check_out(dst[oshift:oshift + total], src[shift:shift + total], 1 / 3)
        assert bool((dst[:oshift] == 5).all()) and bool((dst[oshift + total:] == 5).all())


def test_no_elements(lib):
    assert _call(lib, [], [], 1.0) == 0.0
    empty = [torch.empty(0, device="cuda"), torch.empty((3, 0), dtype=BF, device="cuda")]
    assert _call(lib, empty, empty, 1.0) == 0.0
    zeros = [torch.zeros(100, device="cuda")]
    assert _call(lib, zeros, zeros, 0.0) == 0.0 and bool((zeros[0] == 0).all())


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_ends_of_the_range(lib, dtype):
    """Squares that overflow or vanish in fp32 still give the norm."""
    for level in (1e36, 1e25, 1e15, 1e-15, 1e-25, 3e-38):
        g = _grads([3000, 70], [dtype, dtype], 3, level)
        want = _norm64(g)
        got = _call(lib, g, [torch.empty_like(t) for t in g], math.inf)
        assert abs(got - want) <= (NORM_TOL + U32) * want, (level, got, want)
    # one large element among small ones, and the reverse order of sizes
    g = _grads([5000], [F32], 4, 1e-20)
    g[0][123] = 3e30
    assert abs(_call(lib, g, g, math.inf) - 3e30) <= NORM_TOL * 3e30
    tiny = [torch.full((4,), 2.0 ** -149, device="cuda")]      # subnormals: exactly 2 * 2^-149
    assert _call(lib, tiny, tiny, math.inf) == 2.0 ** -148


def test_not_finite(lib):
    def run(bad, max_norm=1.0):
        g = _grads([4000, 50], [F32, BF], 5)
        g[1][7] = bad
        outs = [torch.empty_like(t) for t in g]
        return _call(lib, g, outs, max_norm), outs

    norm, outs = run(float("inf"))
    assert norm == math.inf and bool((outs[0] == 0).all())
    assert bool(torch.isnan(outs[1][7])) and int(torch.isnan(outs[1]).sum()) == 1
    norm, outs = run(float("-inf"), math.inf)
    assert norm == math.inf and bool(torch.isinf(outs[1][7])) and bool(torch.isfinite(outs[0]).all())
    for m in (1.0, math.inf):
        norm, outs = run(float("nan"), m)
        assert math.isnan(norm) and all(bool(torch.isnan(o).all()) for o in outs)


def test_separate_calls_give_the_same(lib):
    grads = _grads([4097, 31, 9000], [BF, F32, F16], 6)
    a, b = ([torch.empty_like(g) for g in grads] for _ in range(2))
    pa, pb = lib.GradPlan(grads, a), lib.GradPlan(grads, b)
    ws = torch.empty(lib.disco_grad_workspace_bytes(pa.c), dtype=torch.uint8, device="cuda")
    n1, n2 = torch.empty(1, device="cuda"), torch.empty((), device="cuda")
    lib.disco_grad_norm_clip(pa.c, 0.5, n1, ws, grad_scale=0.5)
    lib.disco_grad_norm(pb.c, n2, ws, grad_scale=0.5)
    lib.disco_grad_clip(pb.c, 0.5, n2, grad_scale=0.5)
    torch.cuda.synchronize()
    assert float(n1) == float(n2) and all(torch.equal(u, v) for u, v in zip(a, b))
    only = lib.GradPlan(grads)                                   # the norm needs no outs
    n3 = torch.empty(1, device="cuda")
    lib.disco_grad_norm(only.c, n3, ws, grad_scale=0.5)
    assert float(n3) == float(n1)
    for _ in range(5):                                           # fixed order of summation
        lib.disco_grad_norm(only.c, n3, ws, grad_scale=0.5)
        assert float(n3) == float(n1)


def test_streams_and_graph(lib):
    grads = _grads([200_000, 77], [BF, F32], 7)
    outs = [torch.empty_like(g, dtype=F32) for g in grads]
    want = _norm64(grads)
    plan = lib.GradPlan(grads, outs)
    norm = torch.zeros(1, device="cuda")
    ws = torch.empty(lib.disco_grad_workspace_bytes(plan.c), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    big = torch.zeros(1 << 26, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(4):
            big.add_(1)
        grads[0].mul_(2)                  # arrives late on s
    lib.disco_grad_norm_clip(plan.c, 1.0, norm, ws, stream=s)
    s.synchronize()
    grads64 = _norm64(grads)
    assert grads64 > 1.5 * want and abs(float(norm) - grads64) <= (NORM_TOL + U32) * grads64
    # the call is capturable; a replay sees the gradients of its own time
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.disco_grad_norm_clip(plan.c, 1.0, norm, ws)
    grads[0].div_(4)
    g.replay()
    torch.cuda.synchronize()
    now = _norm64(grads)
    assert abs(float(norm) - now) <= (NORM_TOL + U32) * now
    for o, t in zip(outs, grads):
        _check_out(o, t, min(1.0, 1.0 / now))


def test_offsets_past_32_bits(lib):
    n = (1 << 31) + 4099
    g = torch.zeros(n, dtype=BF, device="cuda")
    g[-1], g[0], g[1 << 31] = 3.0, 4.0, 12.0
    assert _call(lib, [g], [g], 6.5) == 13.0
    assert [float(g[i]) for i in (-1, 0, 1 << 31, 5)] == [1.5, 2.0, 6.0, 0.0]


def test_refusals(lib):
    g = torch.ones(100, device="cuda")
    b = torch.ones(100, dtype=BF, device="cuda")

    def refused(status, text, fn, *args, **kw):
        with pytest.raises(lib.DiscoError) as e:
            fn(*args, **kw)
        assert e.value.status == status and text in str(e.value), str(e.value)

    refused(-1, "CUDA device", lib.GradPlan, [g.cpu()], [g.cpu()])
    refused(-1, "contiguous", lib.GradPlan, [g.view(10, 10).t()])
    refused(-2, "dtype", lib.GradPlan, [g.double()])
    refused(-1, "elements", lib.GradPlan, [g], [g[:50]])
    refused(-1, "outs", lib.GradPlan, [g, b], [g])
    refused(-1, "is None", lib.GradPlan, [None])
    refused(-1, "overlaps", lib.GradPlan, [g[:60], b[:60]], [g[:60], g[40:100].view(-1)])
    refused(-1, "overlaps", lib.GradPlan, [g[:50]], [g[1:51]])
    refused(-1, "overlaps", lib.GradPlan, [g, g], [g, g])
    refused(-1, "overlaps", lib.GradPlan, [g[:50], g[50:]], [g[50:], g[:50]])
    lib.GradPlan([g, g])                                          # read twice: allowed
    plan, only = lib.GradPlan([g], [g]), lib.GradPlan([g])
    norm = torch.zeros(1, device="cuda")
    ws = torch.empty(lib.disco_grad_workspace_bytes(plan.c), dtype=torch.uint8, device="cuda")
    nc = lib.disco_grad_norm_clip
    refused(-1, "max_norm", nc, plan.c, -1.0, norm, ws)
    refused(-1, "max_norm", nc, plan.c, float("nan"), norm, ws)
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        refused(-1, "grad_scale", nc, plan.c, 1.0, norm, ws, grad_scale=scale)
        refused(-1, "grad_scale", lib.disco_grad_norm, plan.c, norm, ws, grad_scale=scale)
    refused(-1, "no out", nc, only.c, 1.0, norm, ws)
    refused(-1, "no out", lib.disco_grad_clip, only.c, 1.0, norm)
    refused(-7, "workspace", nc, plan.c, 1.0, norm, None)
    refused(-7, "workspace", nc, plan.c, 1.0, norm, ws[:-8])
    refused(-1, "elements", nc, plan.c, 1.0, torch.zeros(2, device="cuda"), ws)
    refused(-1, "dtype", nc, plan.c, 1.0, norm.to(BF), ws)
    so = lib.load_library()
    t = (lib.disco_grad_tensor * 1)()
    c = lib.disco_grads()
    t[0].grad, t[0].n, t[0].dtype = g.data_ptr() + 2, 10, lib.DISCO_F32
    assert so.disco_grad_plan(t, 1, ctypes.byref(c)) == -3
    t[0].grad, t[0].out, t[0].out_dtype = b.data_ptr(), b.data_ptr(), lib.DISCO_F32
    t[0].dtype = lib.DISCO_BF16
    assert so.disco_grad_plan(t, 1, ctypes.byref(c)) == -1 and "in place" in lib.disco_last_error()
    host = (ctypes.c_float * 16)()
    t[0].grad, t[0].out, t[0].dtype = ctypes.addressof(host), None, lib.DISCO_F32
    assert so.disco_grad_plan(t, 1, ctypes.byref(c)) == -1 and "device memory" in lib.disco_last_error()
    t[0].n = -1
    assert so.disco_grad_plan(t, 1, ctypes.byref(c)) == -1
    assert so.disco_grad_plan(None, 1, ctypes.byref(c)) == -1 and so.disco_grad_plan(None, 0, None) == -1
    torch.cuda.synchronize()
    assert bool((g == 1).all())
