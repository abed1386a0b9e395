"""fp16 gradients of the integer products over the range of the fp32 scales.

The kernels take a power of two out of a call's scales before scale * integer is rounded to
fp16, so that the largest scale lies in [128, 256) there, and put it back into the sums: to
the bounds of tests/_i8_ops.py a term adds half of fp16's smallest step, 2^-25, at the
largest scale's size, 2^-25 max(scale) / 128 at most, times the other factor."""
import pytest
import torch

from tests import _i8_ops as r
from tests import test_gpu_i8 as t

pytestmark = pytest.mark.gpu

lib = t.lib
HF, F32 = torch.float16, torch.float32

# rows, and grids of whole and odd words; one product whose reductions are split and one with more scales than a block reads at once
SHAPES = [(70, 40, 24, 1), (130, 64, 257, 1), (2, 48, 40, 96), (3, 33, 20, 77), (2, 80, 200, 9001), (300000, 16, 24, 1), (1, 24, 300007, 1)]


def _gradients(lib, shape, dy, q, scale, W, wscale):
    B, Cin, Cout, P = shape
    code = lib.dtype_code(HF)
    dx, dx_ok = r.guarded((B, Cin, P), HF)
    dW, dW_ok = r.guarded((Cout, Cin), HF)
    n = max(f(*shape, code) for f in (lib.disco_matmul_i8_bwd_input_workspace_bytes, lib.disco_matmul_i8_bwd_weight_workspace_bytes))
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    lib.disco_matmul_i8_bwd_input(dy.cuda(), W.cuda(), wscale.cuda(), dx, *shape, ws)
    lib.disco_matmul_i8_bwd_weight(dy.cuda(), q.cuda(), scale.cuda(), dW, *shape, ws)
    dx_ok(), dW_ok()
    assert lib.disco_device_status() == 0
    return dx, dW


def _bound(v, S, D, K, scale):
    return r.grad_bound(v, S, torch.zeros_like(D), K, HF) + 2.0 ** -25 * float(scale.double().abs().max()) / 128 * D


@pytest.mark.parametrize("e", [-100, -30, -18, -8, 8, 16, 26, 100])
@pytest.mark.parametrize("shape", SHAPES, ids=t.ids)
def test_scales_outside_the_types_range(lib, shape, e):
    """Scales times 2^e, with dy of a size that brings the result back as far as it can."""
    B, Cin, Cout, P = shape
    q, scale, W, wscale, dy = t._operands(shape, HF, e)
    g = 2.0 ** max(-8, min(18, -e))
    dy = (dy.float() * g).to(HF)
    scale, wscale = scale * 2.0 ** e, wscale * 2.0 ** e
    dx, dW = _gradients(lib, shape, dy, q, scale, W, wscale)
    most = torch.finfo(HF).max
    for got, (want, S, D), K, s in ((dx, r.bwd_input64(dy, W, wscale), Cout, wscale), (dW, r.bwd_weight64(dy, q, scale), B * P, scale)):
        got, bound = got.double().cpu(), _bound(want, S, D, K, s)
        inside = want.abs() + bound < most  # the rest is infinite in the type
        r.assert_close(torch.where(inside, got, 0.0), torch.where(inside, want, 0.0), bound, "gradient")
        assert bool(((got == torch.where(want > 0, 1.0, -1.0) * float("inf")) | (want.abs() - bound < most) | inside).all())


@pytest.mark.parametrize("shape", [(70, 40, 24, 1), (2, 48, 40, 96)], ids=t.ids)
def test_zeros_and_the_ends_of_fp32(lib, shape):
    """All scales zero, subnormal, or the largest of fp32."""
    B, Cin, Cout, P = shape
    q, scale, W, wscale, dy = t._operands(shape, HF)
    for v in (0.0, 2.0 ** -140, float(torch.finfo(F32).max)):
        dx, dW = _gradients(lib, shape, torch.zeros_like(dy) if v > 1 else dy, q, torch.full_like(scale, v), W, torch.full_like(wscale, v))
        assert bool((dx == 0).all()) and bool((dW == 0).all())


@pytest.mark.parametrize("shape", [(40, 96, 160, 1), (2, 48, 1030, 72), (2, 48, 72, 1165)], ids=t.ids)
def test_streams_graphs_and_spoilt_workspaces(lib, shape):
    """Up to 1024 scales and more: captured and replayed with the workspace spoilt between, and two calls at once."""
    B, Cin, Cout, P = shape
    code = lib.dtype_code(HF)
    runs = []
    for seed in (0, 1):
        q, scale, W, wscale, dy = [v.cuda() for v in t._operands(shape, HF, seed)]
        scale, wscale = scale * 2.0 ** (-20 + 30 * seed), wscale * 2.0 ** (-20 + 30 * seed)
        dx, dW = torch.empty((B, Cin, P), dtype=HF, device="cuda"), torch.empty((Cout, Cin), dtype=HF, device="cuda")
        ws = t._ws(max(f(*shape, code) for f in (lib.disco_matmul_i8_bwd_input_workspace_bytes, lib.disco_matmul_i8_bwd_weight_workspace_bytes)))

        def both(dy=dy, q=q, scale=scale, W=W, wscale=wscale, dx=dx, dW=dW, ws=ws):
            lib.disco_matmul_i8_bwd_input(dy, W, wscale, dx, *shape, ws)
            lib.disco_matmul_i8_bwd_weight(dy, q, scale, dW, *shape, ws)
        both()
        torch.cuda.synchronize()
        runs.append((both, (dx, dW), (dx.clone(), dW.clone()), ws))

    def check():
        torch.cuda.synchronize()
        for _, got, want, ws in runs:
            for a, b in zip(got, want):
                assert torch.equal(a, b)
                a.zero_()
            ws.fill_(255)
        torch.cuda.synchronize()
    check()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(4):
        for s, (both, *_) in zip(streams, runs):
            with torch.cuda.stream(s):
                both()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for both, *_ in runs:
            both()
    for _ in range(3):
        graph.replay()
        check()
    assert lib.disco_device_status() == 0


def test_scales_of_one_call_far_apart(lib):
    """Tokens, and output channels, 2^-24 of the others keep what fp16 holds at the largest one's size."""
    shape = (64, 48, 40, 1)
    B, Cin, Cout, P = shape
    q, scale, W, wscale, dy = t._operands(shape, HF)
    scale[::3] *= 2.0 ** -24
    wscale[1::2] *= 2.0 ** -24
    dx, dW = _gradients(lib, shape, dy, q, scale, W, wscale)
    v, S, D = r.bwd_input64(dy, W, wscale)
    r.assert_close(dx, v, _bound(v, S, D, Cout, wscale), "dx")
    v, S, D = r.bwd_weight64(dy, q, scale)
    r.assert_close(dW, v, _bound(v, S, D, B * P, scale), "dW")
