"""The tests of the 4-bit KV cache, of the reads and of the norms with rotation run
against the bounds-checked build of the library."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = [pytest.mark.gpu, pytest.mark.large]


def test_cache4_and_rope_tests_under_range_checks():
    if os.environ.get("MSA_DEBUG_BOUNDS") == "1":
        pytest.skip("already running against the bounds-checked build")
    from long_context_sparse_landmark_gb300 import build
    build.build(debug_bounds=True)
    env = dict(os.environ, MSA_DEBUG_BOUNDS="1")
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
           "-m", "gpu and not large", "tests/test_gpu_cache4.py", "tests/test_gpu_rope.py"]
    r = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=1500)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-3000:]
    assert "msa bounds check" not in out, "a range check failed"
    assert " passed" in out
