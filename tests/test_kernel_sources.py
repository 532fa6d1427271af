"""Rules that the kernels' sources keep (read as text; nothing runs)."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "differential_attention_03_gb300", "csrc")
HEADERS = sorted(glob.glob(os.path.join(CSRC, "*.cuh")))


def _code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("path", [h for h in HEADERS if "grid_dep_wait()" in _code(h) and os.path.basename(h) != "ptx.cuh"],
                         ids=os.path.basename)
def test_dependents_load_nothing_as_invariant(path):
    """A programmatic dependent runs while the kernel before it may still be writing its inputs: the read-only path, for data
    that do not change while a kernel runs, is not for it, and the compiler may move such loads above the wait."""
    code = _code(path)
    for word in ("__ldg", "__restrict__", ".nc."):
        assert word not in code, (os.path.basename(path), word)
