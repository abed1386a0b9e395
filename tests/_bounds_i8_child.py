"""Runs the 8-bit integer feed-forward's cases on the bounds-checked build of the library.

Started by tests/test_gpu_bounds_i8.py in a process of its own, with
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
    from tests import test_gpu_i8 as t

    assert lib.disco_build_flags() & lib.DISCO_BUILD_DEBUG_BOUNDS, "not the bounds-checked build"
    lib.disco_device_status(clear=True)
    n = 0

    def run(f, *args):
        nonlocal n
        f(lib, *args)
        assert lib.disco_device_status() == 0, args
        n += 1

    for dtype in (torch.float32, torch.bfloat16):
        for shape in t.TOKENS:
            run(t.test_quant_is_the_definition, shape, dtype)
        for shape in t.GLU:
            for outs in ("y", "q", "yx", "yqx"):
                run(t.test_glu, shape, dtype, outs)
            run(t.test_glu_bwd, shape, dtype, 0)
    for shape in t.SHAPES:
        run(t.test_matmul, shape, torch.bfloat16)
        run(t.test_matmul_gradients, shape, torch.float16)
    run(t.test_many_steps_and_tiles, (2, 128, 256, 4112), torch.bfloat16)
    run(t.test_many_steps_and_tiles, (3, 80, 77, 999), torch.bfloat16)
    print(f"bounds-checked: {n} cases clean")
    return 0


if __name__ == "__main__":
    sys.exit(main())
