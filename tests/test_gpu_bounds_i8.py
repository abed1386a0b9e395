"""The 8-bit integer feed-forward on the bounds-checked build (-DDISCO_DEBUG_BOUNDS), in
a child process that loads it: every case right and no range check failed."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_bounds_checked_build_runs_the_feed_forward_clean():
    from sparse_spherical_convolution_gb300 import build
    build.build(debug_bounds=True)
    env = dict(os.environ, DISCO_GB300_BOUNDS_CHECKED="1")
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "_bounds_i8_child.py")], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, (r.stdout[-4000:], r.stderr[-4000:])
    assert "bounds-checked:" in r.stdout and "cases clean" in r.stdout, r.stdout[-2000:]
