"""The suites of the 4-bit linear, the paged cache and its attention again, on the bounds-guard
build libsq_debug.so, in a child process (the binding loads one library per process)."""
import os
import subprocess
import sys

import pytest

from w8a8_quantized_gemm_b200 import build as _b

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SUITES = ["tests/test_gpu_int4.py", "tests/test_gpu_kv.py", "tests/test_gpu_decode_block.py"]


def test_serving_suites_on_the_guarded_build():
    assert os.path.exists(_b.LIB_DEBUG), "libsq_debug.so is not built"
    env = dict(os.environ, SQ_LIB_PATH=_b.LIB_DEBUG)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", *SUITES],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=1800)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout
