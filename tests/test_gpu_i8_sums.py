"""Sums of the 8-bit integer feed-forward on values whose exact sums are known: small integers
times powers of two.

Every product and every partial sum below 2^24 units is exact in fp32 in any order, so where all
of them are, the outputs are the exact values rounded once."""
import pytest
import torch

from tests import _i8_ops as r
from tests import test_gpu_i8 as t

pytestmark = pytest.mark.gpu

lib = t.lib
F32 = torch.float32


def _ints(g, most, shape, dtype=torch.int8):
    return torch.randint(-most, most + 1, shape, generator=g, dtype=torch.int8).to(dtype)


def _pow2(g, lo, shape):
    return 2.0 ** torch.randint(lo, 1, shape, generator=g).float()


# those of many steps and tiles, and one reduction of more than one part's longest
EXACT = [(2, 128, 256, 16400), (2, 128, 256, 16401), (6000, 512, 384, 1), (6001, 515, 391, 1), (1, 1024, 520, 4112), (3, 80, 77, 9999), (1, 4096, 1000, 1),
         (40, 8200, 136, 1), (20000, 512, 256, 1), (2, 515, 300, 9001), (20001, 300, 520, 1), (33000, 2050, 1290, 1), (1, 1100, 2060, 33001)]


@pytest.mark.parametrize("dtype", t.HALF, ids=t.ids)
@pytest.mark.parametrize("shape", EXACT, ids=t.ids)
def test_nothing_is_lost(lib, shape, dtype):
    """Integers up to 15 times 3 times powers of two down to 1/8: 360 units at most to a term, so 46603 terms stay exact."""
    B, Cin, Cout, P = shape
    assert max(B * P, Cin, Cout) * 360 < 2 ** 24
    g = t._gen("exact", shape)
    q, scale = _ints(g, 15, (B, Cin, P)).cuda(), _pow2(g, -3, (B, P)).cuda()
    W, wscale = _ints(g, 15, (Cout, Cin)).cuda(), _pow2(g, -3, (Cout,)).cuda()
    dy = _ints(g, 3, (B, Cout, P), dtype).cuda()
    code = lib.dtype_code(dtype)
    ws = t._ws(max(f(*shape, code) for f in (lib.disco_matmul_i8_workspace_bytes, lib.disco_matmul_i8_bwd_input_workspace_bytes,
                                             lib.disco_matmul_i8_bwd_weight_workspace_bytes)))
    new = lambda *s: torch.full(s, float("nan"), dtype=dtype, device="cuda")  # noqa: E731
    y, dx, dW = new(B, Cout, P), new(B, Cin, P), new(Cout, Cin)
    lib.disco_matmul_i8(q, scale, W, wscale, y, *shape, ws)
    lib.disco_matmul_i8_bwd_input(dy, W, wscale, dx, *shape, ws)
    lib.disco_matmul_i8_bwd_weight(dy, q, scale, dW, *shape, ws)
    for got, want in ((y, r.matmul64(q, scale / 4, W, wscale / 4)[0] * 16), (dx, r.bwd_input64(dy, W, wscale)[0]), (dW, r.bwd_weight64(dy, q, scale)[0])):
        assert torch.equal(want, want.float().double())  # exact in 32 bits: rounded once on the way to the type
        assert torch.equal(got, want.float().to(dtype))
    assert lib.disco_device_status() == 0


@pytest.mark.parametrize("dtype", t.HALF, ids=t.ids)
@pytest.mark.parametrize("shape", [(1 << 21, 2048, 1280, 1), (2, 2048, 1280, (1 << 19) + 8)], ids=t.ids)
def test_long_sums_of_one_sign(lib, shape, dtype):
    """A million tokens or two whose terms are all positive, 1 to 105 units: sums of 32768 tokens are
    exact, their joining adds 64 of them with one rounding each, and dW is rounded once."""
    B, Cin, Cout, P = shape
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randint(1, 8, (B, Cin, P), generator=g, dtype=torch.int8, device="cuda")
    dy = torch.empty((B, Cout, P), dtype=dtype, device="cuda")
    for d in dy.view(-1).split(1 << 28):
        d.copy_(torch.randint(1, 16, d.shape, generator=g, dtype=torch.int8, device="cuda")).mul_(2.0 ** -8)
    scale = torch.full((B, P), 2.0 ** -12, device="cuda")
    dW = torch.empty((Cout, Cin), dtype=dtype, device="cuda")
    ws = t._ws(lib.disco_matmul_i8_bwd_weight_workspace_bytes(*shape, lib.dtype_code(dtype)))
    lib.disco_matmul_i8_bwd_weight(dy, q, scale, dW, *shape, ws)
    want = torch.zeros((Cout, Cin), dtype=torch.float64, device="cuda")
    n = 8192  # tokens whose integer sums are exact in 32 bits
    if P == 1:
        for b in range(0, B, n):
            want += dy[b:b + n, :, 0].float().mul_(2.0 ** 8).t() @ q[b:b + n, :, 0].float()
    else:
        for b in range(B):
            for p in range(0, P, n):
                want += dy[b, :, p:p + n].float().mul_(2.0 ** 8) @ q[b, :, p:p + n].float().t()
    want = (want * 2.0 ** -20).cpu()
    r.assert_close(dW, want, (r.UNIT[dtype] + 64 * r.U32 * 1.001) * want, "dW")
    assert lib.disco_device_status() == 0
