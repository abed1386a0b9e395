"""Runs the channel norm's operators at the ends of small tensors on the
bounds-checked build: rows shorter than a 16-byte word and a little longer, and
odd pixel counts, where the words of a row reach past it.

Started by tests/test_gpu_bounds_edges.py in a process of its own, with
DISCO_GB300_BOUNDS_CHECKED=1.  Every case must match its 64-bit form with a
clean status word.  Prints one line "bounds-checked: <n> cases clean"."""
from __future__ import annotations

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)


def main() -> int:
    assert os.environ.get("DISCO_GB300_BOUNDS_CHECKED") == "1"
    import torch

    import sparse_spherical_convolution_gb300 as lib
    from tests import test_gpu_norm as tn
    from tests._train_ops import TINY, U32, UNIT, assert_close, norm_bwd64

    assert lib.disco_build_flags() & lib.DISCO_BUILD_DEBUG_BOUNDS, "not the bounds-checked build"
    lib.disco_device_status(clear=True)
    rows = [(B, C, 1) for C in (1, 2, 3, 4, 5, 6, 7, 8, 9, 15, 31, 65, 130) for B in (1, 2, 3, 4, 5, 10, 33, 700)]
    grids = [(B, C, P) for B, C in ((1, 1), (2, 3), (1, 40), (2, 70)) for P in (2, 3, 5, 9, 17, 33, 65, 127, 250, 513)]
    n = 0
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        for shape in rows + grids:
            B, C, P = shape
            x, r, w = (tn._randn(s, dtype, 61 + k) for k, s in enumerate((shape, shape, (C,))))
            for group in {0, 1, max(1, C // 2)}:
                tn._check(tn._run(lib, x, r, w, q=True, group=group), x, r, w, group)
            tn._check(tn._run(lib, x, None, None), x, None, None, 0)
            dx, _ = tn._run_bwd(lib, x, r, w, r)
            rx, S, _, _ = norm_bwd64(x, r, w, r, tn.EPS)
            assert_close(dx, rx, (2 * C + 16) * U32 * S + UNIT[dtype] * rx.abs() * 1.01 + TINY[dtype], "dx")
            assert lib.disco_device_status() == 0, (shape, dtype)
            n += 1
        for shape in ((1, 3, 1), (10, 3, 1), (5, 9, 1), (2, 3, 33), (2, 70, 127)):
            tn.test_dequant(lib, shape, dtype)
            assert lib.disco_device_status() == 0, (shape, dtype)
            n += 1
    print(f"bounds-checked: {n} cases clean")
    return 0


if __name__ == "__main__":
    sys.exit(main())
