"""Plain 64-bit forms of the 8-bit integer feed-forward, and the error bounds
its tests use.

Bounds.  u = 2^-24 is fp32's unit roundoff, uo the output type's, both relative
to the value; TINY is half the spacing of the type's subnormals.
  q (quant)  none: the definition's integers.
  scale      amax is exact, one division: u.
  y (matmul) the integer sum is exact within 2^24; two products: (uo + 2 u) |y|.
             Beyond, one rounding at most (truncation: 2 u) for each of the K
             additions and of the accumulator's: 2 K u sum|terms|.
  dx, dW     each term takes scale * integer rounded to the type, uo |term| (and
             TINY of it times the other factor) and u for the product before it;
             sums as above: (uo + 2 (K + 1) u) sum|terms| + uo |value|.
  SiLU       e^-g by the approximate exponential: (2 + 1.173 |g|) ulp, an ulp being
             2 u; the approximate quotient 2 ulp, sum and products under 4 u:
             E(g) = (2 (2 + 1.2 |g|) + 8) u relative.
  GELU       erfc to 4 ulp (8 u) at an argument off by 2 u of itself, which moves
             log erfc(z) by at most (2 z^2 + 2) 2 u, z^2 = g^2 / 2; products 4 u:
             E(g) = (2 (g^2 + 2) + 12) u relative.
  act'       s (1 + g (1 - s)): each of its parts is below 1 + |g| and off by at most
             2 E(g) relative, and g = scale * q is off by u |g|, |act''| <= 1/2:
             (1 + |g|) 3 E(g) absolute.  Phi + g phi: as the sum of its parts, the
             exponential's argument -g^2 / 2 being off by 2 u of itself (g^2 u) and
             the exponential by (2 + 0.6 g^2) ulp: (Phi + |g| phi) (3 E(g) + 4 g^2 u + 4 u).
  q (glu)    127 y / a with y off by e_y (relative, the largest of the token for a):
             127 * 2 (e_y + 4 u) on top of half a unit.
"""
from __future__ import annotations

import math

import torch

from tests._train_ops import TINY, U32, UNIT, assert_close  # noqa: F401

FLOOR = 1e-30


def quant64(x):
    """(q, scale) of x [B, C, P] in 64 bits, where 127 x is exact and the quotient's
    rounding reaches no border that the quotient does not lie on."""
    x = x.double()
    a = x.abs().amax(1, keepdim=True).clamp_min(FLOOR)
    return torch.round(127 * x / a), (a / 127)[:, 0]


def matmul64(q, scale, W, wscale):
    """(y, sum|terms|) for q [B, Cin, P], W [Cout, Cin]."""
    f = wscale.double()[None, :, None] * scale.double()[:, None, :]
    q, W = q.double(), W.double()
    return torch.einsum("oc,bcp->bop", W, q) * f, torch.einsum("oc,bcp->bop", W.abs(), q.abs()) * f.abs()


def bwd_input64(dy, W, wscale):
    """(dx, sum|terms|, sum|dy|) ."""
    w, dy = W.double() * wscale.double()[:, None], dy.double()
    return (torch.einsum("oc,bop->bcp", w, dy), torch.einsum("oc,bop->bcp", w.abs(), dy.abs()),
            dy.abs().sum(1, keepdim=True))


def bwd_weight64(dy, q, scale):
    """(dW, sum|terms|, sum|dy|)."""
    x, dy = q.double() * scale.double()[:, None], dy.double()
    return (torch.einsum("bop,bcp->oc", dy, x), torch.einsum("bop,bcp->oc", dy.abs(), x.abs()),
            dy.abs().sum((0, 2))[:, None])


def matmul_bound(y, S, scale, wscale, K, dtype):
    f = wscale.double()[None, :, None] * scale.double()[:, None, :]
    inexact = (S / f > 2 ** 24).double()
    return (UNIT[dtype] + 2 * U32) * y.abs() + inexact * 2 * K * U32 * S + TINY[dtype]


def grad_bound(v, S, D, K, dtype):
    return UNIT[dtype] * v.abs() + (UNIT[dtype] + 2 * (K + 1) * U32) * S + TINY[dtype] * (1 + D)


def act64(g, act):
    """(act, act', E, bound of act')."""
    if act == 0:
        s = torch.sigmoid(g)
        E = (2 * (2 + 1.2 * g.abs()) + 8) * U32
        return g * s, s * (1 + g * (1 - s)), E, (1 + g.abs()) * 3 * E
    cdf, pdf = torch.special.ndtr(g), torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    E = (2 * (g * g + 2) + 12) * U32
    return g * cdf, cdf + g * pdf, E, (cdf + g.abs() * pdf) * (3 * E + 4 * g * g * U32 + 4 * U32)


def glu64(x, act):
    """(y, relative bound of the unrounded y)."""
    g, v = x.double().chunk(2, 1)
    a, _, E, _ = act64(g, act)
    return a * v, E + 2 * U32


def glu_bwd64(dy, xq, xscale, act, dtype):
    """(dx, bound)."""
    g, v = (xq.double() * xscale.double()[:, None]).chunk(2, 1)
    a, da, E, Ed = act64(g, act)
    dy = dy.double()
    # v and g are products of their own (u each); act(g) moves by |act'| u |g| <= 1.2 u |g|
    bg = (dy * v).abs() * (Ed + 4 * U32 * da.abs())
    bv = dy.abs() * (a.abs() * (E + 3 * U32) + 1.2 * U32 * g.abs())
    dx = torch.cat([dy * v * da, dy * a], 1)
    return dx, torch.cat([bg, bv], 1) + UNIT[dtype] * dx.abs() + TINY[dtype]


def guarded(shape, dtype, device="cuda"):
    """A tensor with 64 elements of a pattern on each side, and the check that they are still there."""
    n = math.prod(shape)
    flat = torch.full((n + 128,), 77, dtype=dtype, device=device)

    def intact():
        assert bool((flat[:64] == 77).all()) and bool((flat[64 + n:] == 77).all()), "written beside the output"
    return flat[64:64 + n].view(shape), intact
