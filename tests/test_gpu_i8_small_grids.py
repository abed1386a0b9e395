"""The gated activation on the smallest odd grids, where the next sample is shorter than a
word: in this process, and on the bounds-checked build in a child process."""
import os
import subprocess
import sys

import pytest

from tests import test_gpu_i8 as t

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
lib = t.lib

# 4 to 14 elements to a sample; a word is 8 of 16 bits or 4 of 32
SHAPES = [(2, 1, 2), (3, 1, 2), (4, 1, 2), (64, 1, 2), (2, 1, 3), (3, 1, 3), (5, 1, 3), (6, 1, 3), (2, 1, 5), (3, 1, 7), (3, 2, 3), (2, 3, 2)]
OUTS = ["y", "q", "yq", "yx", "qx", "yqx"]


@pytest.mark.parametrize("dtype", t.ALL, ids=t.ids)
@pytest.mark.parametrize("shape", SHAPES, ids=t.ids)
@pytest.mark.parametrize("outs", OUTS)
def test_glu(lib, shape, dtype, outs):
    t.test_glu(lib, shape, dtype, outs)


@pytest.mark.parametrize("dtype", t.ALL, ids=t.ids)
@pytest.mark.parametrize("shape", SHAPES, ids=t.ids)
def test_glu_bwd_and_quant(lib, shape, dtype):
    for act in (0, 1):
        t.test_glu_bwd(lib, shape, dtype, act)
    t.test_quant_is_the_definition(lib, shape, dtype)


def test_bounds_checked_build_runs_them_clean():
    from sparse_spherical_convolution_gb300 import build
    build.build(debug_bounds=True)
    env = dict(os.environ, DISCO_GB300_BOUNDS_CHECKED="1")
    r = subprocess.run([sys.executable, "-m", "tests.test_gpu_i8_small_grids"], cwd=ROOT, env=env, capture_output=True, text=True,
                       timeout=1200)
    assert r.returncode == 0, (r.stdout[-4000:], r.stderr[-4000:])
    assert f"bounds-checked: {len(SHAPES) * 3 * (len(OUTS) + 3)} cases clean" in r.stdout, r.stdout[-2000:]


def main():
    import sparse_spherical_convolution_gb300 as d
    assert d.disco_build_flags() & d.DISCO_BUILD_DEBUG_BOUNDS, "not the bounds-checked build"
    d.disco_device_status(clear=True)
    n = 0
    for dtype in t.ALL:
        for shape in SHAPES:
            calls = [(t.test_glu, outs) for outs in OUTS] + [(t.test_glu_bwd, 0), (t.test_glu_bwd, 1), (t.test_quant_is_the_definition,)]
            for f, *more in calls:
                f(d, shape, dtype, *more)
                assert d.disco_device_status() == 0, (f, shape, dtype, more)
                n += 1
    print(f"bounds-checked: {n} cases clean")


if __name__ == "__main__":
    main()
