"""One training step of a residual stack of DISCO convolutions on the sphere.

    python examples/residual_stack.py [--steps 5] [--layers 3] [--channels 64] [--nlat 33] [--nlon 64]

Layer l adds its convolution to the residual stream and normalises the sum:

    h_l = h_{l-1} + y_{l-1},   n_l = rms_norm(h_l) weight_l,   y_l = W_l * n_l

The norm's forward writes h_l over the residual stream's next buffer, n_l for
the convolution, and n_l in 8 bits with scales.  n_l itself is dropped: the
weight gradient restores it from the 8-bit copy, so a layer keeps 1 byte of n_l
and 2 of h_l for each element.  After the backward pass the norm over all
gradients is taken and the gradients go, clipped, into one flat fp32 buffer,
from which the fp32 weights are updated (plain SGD).  The loss is the mean
square distance of the last norm to a target.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import sparse_spherical_convolution_gb300 as d  # noqa: E402

EPS, GROUP = 1e-5, 32


class Stack:
    def __init__(self, layers: int, channels: int, nlat: int, nlon: int, batch: int, seed: int = 0):
        self.L, self.C, self.B, self.P = layers, channels, batch, nlat * nlon
        grid = (nlat, nlon, 1)
        self._psi = d.Psi(grid, grid, 1, 3, 3 * math.pi / (nlat - 1))  # owns the memory that psi points to
        self.psi = self._psi.c
        self.K = self.psi.K
        B, C, P, K, bf = self.B, self.C, self.P, self.K, torch.bfloat16
        g = torch.Generator(device="cuda").manual_seed(seed)
        sizes = [C * C * K] * layers + [C] * (layers + 1)
        # fp32 weights and clipped gradients, each in one flat buffer; bf16 views of the weights for the kernels
        self.master = torch.cat([torch.randn(n, generator=g, device="cuda") / math.sqrt(C * K) if n > C else
                                 torch.ones(n, device="cuda") for n in sizes])
        self.clipped = torch.empty_like(self.master)
        # each weight a 16-byte aligned tensor of its own
        self.weights = [torch.empty(n, dtype=bf, device="cuda") for n in sizes]
        self.grads = [torch.empty(n, dtype=bf, device="cuda") for n in sizes]
        self.sizes = sizes
        new = lambda dt=bf: torch.empty((B, C, P), dtype=dt, device="cuda")  # noqa: E731
        self.h = [new() for _ in range(layers + 1)]
        self.q = [new(torch.float8_e4m3fn) for _ in range(layers)]
        self.scale = [torch.empty((B, -(-C // GROUP), P), device="cuda") for _ in range(layers)]
        self.n, self.y, self.out = new(), new(), new()
        self.dh, self.dn, self.dy = new(), new(), new()
        self.loss_grad = new()
        code = d.dtype_code(bf)
        ws = max(d.disco_fused_conv_workspace_bytes(self.psi, B, C, C, code),
                 d.disco_fused_conv_bwd_input_workspace_bytes(self.psi, B, C, code),
                 d.disco_fused_conv_bwd_weight_workspace_bytes(self.psi, B, C, C, code),
                 d.disco_rms_norm_bwd_workspace_bytes(B, C, P, code))
        self.ws = torch.empty(max(ws, 256), dtype=torch.uint8, device="cuda")
        self.plan = d.GradPlan(self.grads, list(self.clipped.split(sizes)))
        self.norm = torch.empty((), device="cuda")
        self.grad_ws = torch.empty(d.disco_grad_workspace_bytes(self.plan.c), dtype=torch.uint8, device="cuda")
        self._cast()

    def _cast(self):
        for w, m in zip(self.weights, self.master.split(self.sizes)):
            w.copy_(m)

    def forward(self, x):
        """The last norm of the stack for x [B, C, P] (bf16)."""
        B, C, P, L = self.B, self.C, self.P, self.L
        W, gain = self.weights[:L], self.weights[L:]
        self.h[0].copy_(x)
        for l in range(L):
            if l == 0:
                d.disco_rms_norm(self.h[0], None, gain[0], EPS, None, self.n, B, C, P, q=self.q[0], scale=self.scale[0], group=GROUP)
            else:
                d.disco_rms_norm(self.y, self.h[l - 1], gain[l], EPS, self.h[l], self.n, B, C, P, q=self.q[l],
                                 scale=self.scale[l], group=GROUP)
            d.disco_fused_conv(self.psi, self.n, W[l], self.y, B, C, C, self.ws)
        d.disco_rms_norm(self.y, self.h[L - 1], gain[L], EPS, self.h[L], self.out, B, C, P)
        return self.out

    def backward(self, dout):
        """All gradients for the gradient of the last norm."""
        B, C, P, L = self.B, self.C, self.P, self.L
        W, gain, g = self.weights[:L], self.weights[L:], self.grads
        # dh: the gradient of the residual stream, which is also that of the convolution's output
        d.disco_rms_norm_bwd(dout, self.h[L], gain[L], None, EPS, self.dh, g[2 * L], B, C, P, self.ws)
        for l in reversed(range(L)):
            d.disco_dequant_e4m3(self.q[l], self.scale[l], self.n, B, C, P, GROUP)
            d.disco_fused_conv_bwd_weight(self.psi, self.n, self.dh, g[l], B, C, C, self.ws)
            d.disco_fused_conv_bwd_input(self.psi, self.dh, W[l], self.dn, B, C, C, self.ws)
            d.disco_rms_norm_bwd(self.dn, self.h[l], gain[l], self.dh, EPS, self.dh, g[L + l], B, C, P, self.ws)

    def step(self, x, target, lr: float, max_norm: float):
        """One update; the loss before it and the gradients' norm, as device scalars."""
        diff = self.forward(x).float() - target
        loss = diff.square().mean()
        self.loss_grad.copy_(diff.mul_(2 / diff.numel()))
        self.backward(self.loss_grad)
        d.disco_grad_norm_clip(self.plan.c, max_norm, self.norm, self.grad_ws)
        self.master.sub_(self.clipped, alpha=lr)
        self._cast()
        return loss, self.norm.clone()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=5)
    ap.add_argument("--layers", type=int, default=3)
    ap.add_argument("--channels", type=int, default=64)
    ap.add_argument("--batch", type=int, default=2)
    ap.add_argument("--nlat", type=int, default=33)
    ap.add_argument("--nlon", type=int, default=64)
    ap.add_argument("--lr", type=float, default=1.0)
    ap.add_argument("--max-norm", type=float, default=0.2,
                    help="limit of the gradients' norm; at the default sizes it starts at 0.25")
    a = ap.parse_args(argv)
    s = Stack(a.layers, a.channels, a.nlat, a.nlon, a.batch)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((s.B, s.C, s.P), generator=g, device="cuda").bfloat16()
    target = torch.randn((s.B, s.C, s.P), generator=g, device="cuda")
    losses = []
    for k in range(a.steps):
        loss, norm = s.step(x, target, a.lr, a.max_norm)
        losses.append(float(loss))
        print(f"step {k}: loss {losses[-1]:.5f}, gradient norm {float(norm):.4f}")
    if d.disco_device_status() != 0:
        raise RuntimeError("a bounded wait timed out")
    return losses


if __name__ == "__main__":
    main()
