"""Gradient lists longer than one launch takes (1000 tensors), with empty
tensors among them or nothing else, and norms whose unscaled value lies outside
fp32's range.

Bound of the norm.  All sums are fp32 and all terms positive, so the sum of
squares is off by at most one rounding (2^-24) for each addition on a term's way
to the result.  These lists run in two launches or more: a chunk has 256 elements,
8 to a lane in two chains of 4, and a warp takes at most 3 of a launch's (fewer than
9728 and one for each tensor, over up to 4864 warps): 12 additions, 1 of the two
chains, 5 over the lanes, 7 over the warps, fewer than 8 over a thread's rows of
partial sums, again 5 and 7.  Below 48, which is 24 roundings of the root; the
root, the scale and its power of two add 3.
"""
import math

import pytest
import torch

from tests._train_ops import TINY, U32, UNIT

pytestmark = pytest.mark.gpu
F32, BF, F16 = torch.float32, torch.bfloat16, torch.float16
NORM_TOL = 27 * U32


@pytest.fixture(scope="module")
def lib():
    from sparse_spherical_convolution_gb300 import build
    build.build()
    import sparse_spherical_convolution_gb300 as d
    d.disco_device_status(clear=True)
    return d


def _norm64(grads):
    flat = torch.cat([g.double().flatten() for g in grads]) if grads else torch.zeros(1, dtype=torch.float64)
    return float(flat.square().sum().sqrt())


def _lists(count, seed):
    """count gradients of three types, every fifth empty, of 1 to 300 elements."""
    g = torch.Generator().manual_seed(seed)
    sizes = [0 if i % 5 == 2 else 1 + (37 * i) % 300 for i in range(count)]
    return [(1e-2 * torch.randn(n, generator=g)).to((F32, BF, F16)[i % 3]).cuda() for i, n in enumerate(sizes)]


def _buffers(lib, plan):
    return (torch.full((1,), -1.0, device="cuda"),
            torch.full((lib.disco_grad_workspace_bytes(plan.c),), 0xFF, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("in_place", [False, True], ids=["f32 out", "in place"])
@pytest.mark.parametrize("count", [999, 1000, 1001, 2000, 2103])
def test_lists_of_several_launches(lib, count, in_place):
    keep = _lists(count, count)
    want = _norm64(keep)
    for max_norm, scale in ((0.37 * want, 1.0), (0.2 * want, 0.25), (2 * want, 0.5)):
        factor = scale if scale * want <= max_norm else max_norm / want
        results = []
        for joint in (True, False):
            grads = [g.clone() for g in keep]
            outs = grads if in_place else [torch.full_like(g, 9.0, dtype=F32) for g in grads]
            plan = lib.GradPlan(grads, outs)
            norm, ws = _buffers(lib, plan)
            if joint:
                lib.disco_grad_norm_clip(plan.c, max_norm, norm, ws, grad_scale=scale)
            else:
                lib.disco_grad_norm(plan.c, norm, ws, grad_scale=scale)
                lib.disco_grad_clip(plan.c, max_norm, norm, grad_scale=scale)
            torch.cuda.synchronize()
            assert abs(float(norm) - scale * want) <= NORM_TOL * scale * want
            for o, g in zip(outs, keep):
                w = g.double() * factor
                tol = (NORM_TOL + 5 * U32 + UNIT[o.dtype] * 1.01) * w.abs() + TINY[o.dtype] * 1.01
                assert bool(((o.double() - w).abs() <= tol).all())
            results.append((norm, outs))
        assert float(results[0][0]) == float(results[1][0])
        assert all(torch.equal(a, b) for a, b in zip(results[0][1], results[1][1]))


@pytest.mark.parametrize("count", [1, 1000, 1001, 2103])
def test_lists_of_empty_tensors(lib, count):
    """No elements: the norm is 0, whichever call computes it."""
    empty = [torch.empty(0, dtype=(F32, BF, F16)[i % 3], device="cuda") for i in range(count)]
    plan = lib.GradPlan(empty, empty)
    norm, ws = _buffers(lib, plan)
    lib.disco_grad_norm_clip(plan.c, 1.0, norm, ws)
    assert float(norm) == 0.0
    norm.fill_(-1.0)
    lib.disco_grad_norm(plan.c, norm, ws)
    assert float(norm) == 0.0
    lib.disco_grad_clip(plan.c, 1.0, norm)
    torch.cuda.synchronize()


@pytest.mark.parametrize("count", [1001, 2103])
def test_one_tensor_with_elements_at_the_end(lib, count):
    grads = [torch.empty(0, device="cuda") for _ in range(count - 1)] + [torch.tensor([3.0, 4.0], device="cuda")]
    plan = lib.GradPlan(grads, grads)
    norm, ws = _buffers(lib, plan)
    lib.disco_grad_norm_clip(plan.c, 2.5, norm, ws)
    assert float(norm) == 5.0 and grads[-1].tolist() == [1.5, 2.0]


# gradients (value, elements, type), grad_scale: the norm itself lies in fp32's
# range, before the scale it is above it or among its subnormals
SCALED = [
    (3e38, 4, BF, 2.0 ** -16), (3e38, 4, F32, 2.0 ** -16), (3e38, 70_000, F32, 2.0 ** -100), (1e38, 9_000, BF, 2.0 ** -149),
    (2.0 ** -148, 3, F32, 2.0 ** 16), (2.0 ** -148, 3, F32, 2.0 ** 100), (1e-40, 70_000, F32, 2.0 ** 127), (65504.0, 1000, F16, 2.0 ** 100),
    (1.0, 5000, F32, 2.0 ** -149), (1.0, 70_000, BF, 2.0 ** 119),
]


@pytest.mark.parametrize("value,n,dtype,scale", SCALED, ids=lambda v: f"{v:.3g}" if isinstance(v, (int, float)) else str(v)[6:])
def test_norm_outside_the_range_before_its_scale(lib, value, n, dtype, scale):
    """Lists of one launch and of two (70,000 elements; there each thread adds
    at most 3 chunks too)."""
    g = [torch.full((n,), value).to(dtype).cuda()]
    want = scale * math.sqrt(n) * float(g[0][0].double())
    tiny = TINY[F32] * 1.01                            # a norm among the subnormals is rounded to their spacing
    for joint in (True, False):
        outs = [torch.empty((n,), dtype=F32, device="cuda")]
        plan = lib.GradPlan(g, outs)
        norm, ws = _buffers(lib, plan)
        if joint:
            lib.disco_grad_norm_clip(plan.c, math.inf, norm, ws, grad_scale=scale)
            w = g[0].double() * scale
            assert bool(((outs[0].double() - w).abs() <= U32 * w + tiny).all())
        else:
            lib.disco_grad_norm(plan.c, norm, ws, grad_scale=scale)
        assert abs(float(norm) - want) <= NORM_TOL * want + tiny, (float(norm), want)


# gradients (value, elements, type), grad_scale and max_norm: the factor, or a
# quotient on its way, lies near or below the smallest normal fp32 value 2^-126
SMALL_FACTORS = [
    (1e30, 4, F32, 1.0, 1e-10), (1e33, 4, F32, 2.0 ** 14, 1e-6), (3e38, 1, BF, 1.0, 1e-6), (3e38, 2, F32, 2.0 ** -16, 1.0),
    (1e38, 70_000, F32, 2.0 ** -30, 1e-20), (2.0 ** 127, 1, F32, 1.0, 2.0 ** -120), (6e4, 9, F16, 2.0 ** 100, 1e-30),
    (1e20, 5, F32, 1.0, 0.0), (1e-30, 5, F32, 2.0 ** 20, 1e-36),
]


@pytest.mark.parametrize("value,n,dtype,scale,max_norm", SMALL_FACTORS,
                         ids=lambda v: f"{v:.3g}" if isinstance(v, (int, float)) else str(v)[6:])
def test_small_factors(lib, value, n, dtype, scale, max_norm):
    """Clipped gradients keep fp32's relative accuracy down to its subnormals,
    however far their norm is above max_norm: the factor's 3 operations, a
    second product, and the norm's own error."""
    g = [torch.cat([torch.full((n,), value), torch.tensor([value / 1024, -value / 7, 0.0])]).to(dtype).cuda()]
    N = scale * float(g[0].double().norm())
    assert N > max_norm
    want = g[0].double() * (scale * max_norm / N)
    for joint in (True, False):
        for odt in (F32, dtype):
            outs = [torch.empty_like(g[0], dtype=odt)]
            plan = lib.GradPlan(g, outs)
            norm, ws = _buffers(lib, plan)
            if joint:
                lib.disco_grad_norm_clip(plan.c, max_norm, norm, ws, grad_scale=scale)
            else:
                lib.disco_grad_norm(plan.c, norm, ws, grad_scale=scale)
                lib.disco_grad_clip(plan.c, max_norm, norm, grad_scale=scale)
            assert abs(float(norm) - N) <= NORM_TOL * N
            # TINY[odt]: half a subnormal step of the type; fp32's own for the product before it
            tol = (NORM_TOL + 6 * U32 + UNIT[odt] * 1.01) * want.abs() + 1.01 * (TINY[odt] + 2 * TINY[F32])
            assert bool(((outs[0].double() - want).abs() <= tol).all()), (outs[0][:1], want[:1])


def test_norm_of_a_hundred_million_elements(lib):
    """Chunks of 8192 elements, 128 to each of a lane's two chains, and at most
    ceil(chunks / 4864) chunks to a warp: so many additions and 36 of the joins
    on a term's way, half of that in the root.  A lost chunk would show."""
    n = 100_000_007
    g = torch.randn(n, generator=torch.Generator(device="cuda").manual_seed(8), device="cuda").bfloat16()
    chunks = -(-n // 8192)
    tol = ((-(-chunks // 4864) * 128 + 36) / 2 + 3) * U32
    want = _norm64([g])
    assert math.sqrt(1 - 8192 / n) < 1 - tol
    plan = lib.GradPlan([g])
    norm, ws = _buffers(lib, plan)
    lib.disco_grad_norm(plan.c, norm, ws)
    assert abs(float(norm) - want) <= tol * want, float(norm) / want - 1


def test_norm_and_workspace_apart_from_the_gradients(lib):
    """A norm or workspace inside a gradient, an out or one another is refused;
    beside them it is taken, and so is a workspace in the outs of a call that
    does not write them."""
    flat, dst = torch.ones(20_000, device="cuda"), torch.zeros(20_000, device="cuda")
    need = lib.disco_grad_workspace_bytes(lib.GradPlan([flat]).c)
    assert need % 16 == 0 and need < 8_000 * 4
    grads, outs = [flat[:100], flat[100:9_000]], [dst[:100], dst[100:9_000]]
    plan, same = lib.GradPlan(grads, outs), lib.GradPlan(grads, grads)
    norm, ws = _buffers(lib, plan)

    def refused(text, fn, *args):
        with pytest.raises(lib.DiscoError) as e:
            fn(*args)
        assert e.value.status == -1 and text in str(e.value), str(e.value)

    def words(t, first):                                 # a workspace from element `first` of t
        return t[first:first + need // 4].view(torch.uint8)

    joint, alone, clip = lib.disco_grad_norm_clip, lib.disco_grad_norm, lib.disco_grad_clip
    refused("norm overlaps gradient 0", joint, plan.c, 1.0, flat[99:100], ws)
    refused("norm overlaps gradient 1", alone, plan.c, flat[100:101], ws)
    refused("norm overlaps the out of gradient 1", joint, plan.c, 1.0, dst[8_999:9_000], ws)
    refused("norm overlaps the out of gradient 0", clip, plan.c, 1.0, dst[:1])
    refused("norm overlaps the out of gradient 0", clip, same.c, 1.0, flat[:1])
    refused("the workspace overlaps gradient 1", joint, plan.c, 1.0, norm, words(flat, 8_996))
    refused("the workspace overlaps gradient 0", alone, plan.c, norm, words(flat, 0))
    refused("the workspace overlaps the out of gradient 1", joint, plan.c, 1.0, norm, words(dst, 8_000))
    for fn, args in ((joint, (plan.c, 1.0)), (alone, (plan.c,))):
        refused("norm overlaps the workspace", fn, *args, ws.view(torch.float32)[need // 4 - 1:], ws)
    want = math.sqrt(9_000)
    joint(plan.c, 1.0, flat[9_000:9_001], words(flat, 9_004))
    assert abs(float(flat[9_000]) - want) <= NORM_TOL * want
    alone(plan.c, dst[9_000:9_001], words(dst, 0))
    assert abs(float(dst[9_000]) - want) <= NORM_TOL * want
    clip(plan.c, 1.0, flat[9_000:9_001])
    assert bool(((dst[:9_000] - 1 / want).abs() <= (NORM_TOL + 6 * U32) / want).all())
