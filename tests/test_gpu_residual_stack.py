"""The example's training step: its gradients against the loss's differences,
and a loss that falls."""
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from sparse_spherical_convolution_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import residual_stack
    return residual_stack


def test_gradients_match_differences_of_the_loss(example):
    """Along the gradient itself the loss changes by |g|^2 a unit step.  bf16
    activations and an 8-bit copy (relative rounding 2^-8 and 2^-4, averaged over
    33 x 64 x 2 pixels) leave the gradient's direction within a few percent, and
    central differences over a 5% change of the loss have a second-order error of
    the same size: 15% in all."""
    s = example.Stack(2, 64, 33, 64, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((s.B, s.C, s.P), generator=g, device="cuda").bfloat16()
    target = torch.randn((s.B, s.C, s.P), generator=g, device="cuda")

    def loss_at(master):
        s.master.copy_(master)
        s._cast()
        return float((s.forward(x).float() - target).square().mean())

    start = s.master.clone()
    s.step(x, target, 0.0, math.inf)          # clipped = the gradients themselves
    grad, n2 = s.clipped.clone(), float(s.clipped.double().square().sum())
    assert abs(float(s.norm) ** 2 - n2) <= 1e-5 * n2
    step = 0.05 * loss_at(start) / n2
    diff = (loss_at(start + step * grad) - loss_at(start - step * grad)) / (2 * step)
    assert abs(diff - n2) <= 0.15 * n2, (diff, n2)


def test_loss_falls_and_clipping_holds(example):
    losses = example.main(["--steps", "6", "--layers", "2"])
    assert losses[-1] < losses[0] and all(math.isfinite(v) for v in losses)
    s = example.Stack(2, 64, 33, 64, 2)
    x = torch.randn((s.B, s.C, s.P), device="cuda").bfloat16()
    _, norm = s.step(x, torch.randn((s.B, s.C, s.P), device="cuda"), 0.1, 1e-3)
    assert float(norm) > 1e-3 and abs(float(s.clipped.norm()) - 1e-3) <= 1e-6
