"""The bounds-check build on the rotary, cache append, tree decode and cache keep kernels.

Every TMA coordinate, tensor-memory address and global store that they check is checked on the small
cases of their parity tests, in a child process with DIFFATTN_DEBUG=1: those tests read the device
status after their kernels, so that a failed check fails them.
"""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SMALL = ("rope_matches or append or tree_v1_matches or tree_v2_matches or blind or sees_nothing or same_bits or many_tiles "
         "or keep or speculative or chain_of_drafts or graph or references_move or non_finite or underflow")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from differential_attention_03_gb300 import build
    build.build(bounds=True)


def test_cache_cases_pass_under_bounds_checks():
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "tests/test_gpu_cache.py",
           "tests/test_gpu_cache_edges.py", "-k", SMALL]
    r = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, DIFFATTN_DEBUG="1"), capture_output=True, text=True, timeout=1200)
    tail = (r.stdout + r.stderr)[-4000:]
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and " failed" not in r.stdout, tail
    assert int(r.stdout.rsplit(" passed", 1)[0].split()[-1]) >= 150, tail
