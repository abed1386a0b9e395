"""Plain 64-bit forms of the channel norm, its gradient, the 8-bit copy and
gradient clipping, and the error bounds their tests use.

Bounds.  u = 2^-24 is fp32's unit roundoff, uo the output type's.  All sums in
question run over C (or B*P) fp32 terms in some order, so a sum of n terms is
off by at most n u sum|terms|.
  y      relative: the sum of squares (all positive) by C u, its root by half
         of that, and fewer than 8 further roundings.
  scale  as y, and 4 more roundings.
  dx     the terms are r |g|, r |n| mean|g n| and |dh|; mean(g n) is off by
         C u mean|g n| and each n by (C/2 + 8) u: 2 C + 16 roundings of the sum
         of the terms.
  dw     N = B P terms: (N + C/2 + 8) u sum|terms|.
"""
from __future__ import annotations

import torch

U32 = 2.0 ** -24
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# half the spacing of the type's subnormals
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def norm64(x, residual, weight, eps):
    """(h, y) in 64 bits; x [B, C, P]."""
    h = x.double()
    if residual is not None:
        h = h + residual.double()
    w = torch.ones(x.shape[1], dtype=torch.float64) if weight is None else weight.double()
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * w[None, :, None]
    return h, y


def quant64(y, group):
    """(scale, y * 448 / m) in 64 bits: what q rounds."""
    B, C, P = y.shape
    G = group if 0 < group < C else C
    scale, v = [], torch.empty_like(y)
    for c in range(0, C, G):
        m = y[:, c:c + G].abs().amax(1).clamp_min(1e-30)
        scale.append(m / 448)
        v[:, c:c + G] = y[:, c:c + G] * 448 / m[:, None]
    return torch.stack(scale, 1), v


def norm_bwd64(dy, h, weight, dh, eps):
    """(dx, sum|terms| of dx, dweight, sum|terms| of dweight) in 64 bits."""
    dy, h = dy.double(), h.double()
    w = torch.ones(h.shape[1], dtype=torch.float64) if weight is None else weight.double()
    r = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    n, g = h * r, dy * w[None, :, None]
    dx = r * (g - n * (g * n).mean(1, keepdim=True))
    S = r * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if dh is not None:
        dx, S = dx + dh.double(), S + dh.double().abs()
    return dx, S, (dy * n).sum((0, 2)), (dy * n).abs().sum((0, 2))


def assert_close(got, want, bound, what):
    """|got - want| <= bound everywhere, and NaN / infinities in the same places."""
    got, want = got.double().cpu(), want.double()
    bad = torch.isnan(want) != torch.isnan(got)
    fin = torch.isfinite(want)
    bad |= ~fin & ~torch.isnan(want) & (got != want)
    bad |= fin & ~((got - want).abs() <= bound)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        b = torch.as_tensor(bound).broadcast_to(want.shape)[i]
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got {got[i].item()!r}, "
                             f"want {want[i].item()!r} within {float(b):.3e}")


def e4m3_half_step(v):
    """Half the spacing of e4m3 values around v."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)))
    return torch.exp2(e - 4)
