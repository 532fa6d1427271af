"""The bounds-check build on the block's kernels: products, element-wise backward, norms.

Every TMA coordinate, bulk copy, tensor-memory address and global store that they check is checked on cases of
their parity tests, in a child process with DIFFATTN_DEBUG=1: those tests read the device status after their
kernels, so that a failed check fails them.
"""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CASES = "test_linear or test_gated or test_norm or poisoned or rows_nan or see_each_other or graphs or block_and_its_gradients"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from differential_attention_03_gb300 import build
    build.build(bounds=True)


def test_block_cases_pass_under_bounds_checks():
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "tests/test_gpu_block.py",
           "tests/test_gpu_block_edges.py", "-k", CASES]
    r = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, DIFFATTN_DEBUG="1"), capture_output=True, text=True, timeout=1200)
    tail = (r.stdout + r.stderr)[-4000:]
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and " failed" not in r.stdout, tail
    assert int(r.stdout.rsplit(" passed", 1)[0].split()[-1]) >= 300, tail
