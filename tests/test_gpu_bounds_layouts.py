"""The bounds-check build on the products' layouts and on long contractions in fp32: every TMA coordinate, tensor-memory
column and global store that they check, in a child process with DIFFATTN_DEBUG=1.  Those tests read the device status after
their kernels, so that a failed check fails them.
"""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_layouts_pass_under_bounds_checks():
    from differential_attention_03_gb300 import build
    build.build(bounds=True)
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "tests/test_gpu_block_layouts.py",
           "tests/test_gpu_linear_fp32.py", "tests/test_gpu_gelu_tail.py"]
    r = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, DIFFATTN_DEBUG="1"), capture_output=True, text=True, timeout=1200)
    tail = (r.stdout + r.stderr)[-4000:]
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and " failed" not in r.stdout, tail
    assert int(r.stdout.rsplit(" passed", 1)[0].split()[-1]) >= 90, tail
