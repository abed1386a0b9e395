"""Runs the training operators' cases on the bounds-checked build of the library.

Started by tests/test_gpu_bounds_train.py in a process of its own, with
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
    from tests import test_gpu_grad as tg
    from tests import test_gpu_norm as tn

    assert lib.disco_build_flags() & lib.DISCO_BUILD_DEBUG_BOUNDS, "not the bounds-checked build"
    lib.disco_device_status(clear=True)
    n = 0
    small = [s for s in tn.SHAPES + tn.LONG if s[0] * s[1] * s[2] <= 600_000]
    for dtype in (torch.float32, torch.bfloat16):
        for shape in small:
            tn.test_norm_matches_64_bits(lib, shape, dtype)
            tn.test_gradient_matches_64_bits(lib, shape, dtype)
            assert lib.disco_device_status() == 0, shape
            n += 1
        for shape in ((5, 100, 1), (2, 33, 7), (3, 20, 1001), (2, 48, 130)):
            tn.test_dequant(lib, shape, dtype)
            assert lib.disco_device_status() == 0, shape
            n += 1
    for name in tg.LISTS:
        tg.test_norm_and_clip(lib, name, "f32 out")
        assert lib.disco_device_status() == 0, name
        n += 1
    print(f"bounds-checked: {n} cases clean")
    return 0


if __name__ == "__main__":
    sys.exit(main())
