"""The parity tests of the gated delta rule and of the root-mean-square norm
once more under the index-checked library (libm3_debug.so): every access of
their kernels is compared with its buffer's extent, and the conftest fixture
fails any test whose kernels recorded a failed check.  A child process, since
the package picks its library at import."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("path", ["tests/test_delta_gpu.py", "tests/test_delta_many_chunks_gpu.py",
                                  "tests/test_delta_streams_gpu.py", "tests/test_norm_gpu.py", "tests/test_norm_odd_gpu.py"])
def test_parity_under_the_checked_library(path):
    env = dict(os.environ, M3_DEBUG_BOUNDS="1", PYTHONPATH=ROOT)
    code = ("import selective_state_space_m3_b200 as m3\n"
            "assert m3.LIB_PATH.endswith('libm3_debug.so')\n"
            "import sys, pytest\n"
            f"sys.exit(pytest.main(['-q', '-x', '-p', 'no:cacheprovider', '{path}']))\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env, cwd=ROOT, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and "failed" not in r.stdout, r.stdout[-2000:]
