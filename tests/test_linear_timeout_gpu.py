"""Waits of the product kernels that run out on the GPU: the debug-bounds build leaves one
copy out, and the call must report MOE_DEVERR_TIMEOUT, return, and leave the context
usable.  The library is chosen once per process, so the cases run in a child process."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_waits_that_run_out_are_reported_and_the_context_recovers():
    env = dict(os.environ, MOE_INT4_DEBUG_BOUNDS="1")
    env.pop("MOE_LINEAR_DEBUG_SKIP_LINE", None)
    r = subprocess.run([sys.executable, os.path.join(HERE, "linear_timeout_check.py")], env=env,
                       capture_output=True, text=True, timeout=300)
    print(r.stdout)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "linear timeouts: all cases reported and recovered" in r.stdout
