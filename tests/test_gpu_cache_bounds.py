"""The tests of the 8-bit KV cache run against the bounds-checked build of the
library: every range check of the cache's kernels holds, and a page or length
that the kernels refuse is the only thing that sets the status word."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = [pytest.mark.gpu, pytest.mark.large]


def test_cache_tests_under_range_checks():
    if os.environ.get("MSA_DEBUG_BOUNDS") == "1":
        pytest.skip("already running against the bounds-checked build")
    from long_context_sparse_landmark_gb300 import build
    build.build(debug_bounds=True)
    env = dict(os.environ, MSA_DEBUG_BOUNDS="1")
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
           "-m", "gpu and not large", "tests/test_gpu_cache.py"]
    r = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=1500)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-3000:]
    assert "msa bounds check" not in out, "a range check failed"
    assert " passed" in out
