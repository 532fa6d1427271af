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


KERNEL = re.compile(r"__global__.*?\n}\n", re.S)


@pytest.mark.parametrize("path", [h for h in HEADERS if "tmem_alloc" in _code(h) and os.path.basename(h) != "ptx.cuh"],
                         ids=os.path.basename)
def test_dependents_start_when_tensor_memory_is_held(path):
    """A kernel lets its dependents start only when its CTAs hold their tensor memory: a dependent takes its own before it
    waits, and neither tcgen05.alloc nor griddepcontrol.wait has a time limit."""
    kernels = [k for k in KERNEL.findall(_code(path)) if "tmem_alloc" in k]
    assert kernels
    for k in kernels:
        if "grid_dep_launch_dependents()" in k:
            taken = max(m.start() for m in re.finditer("tmem_alloc", k))
            held = k.index("__syncthreads()", taken)
            assert k.index("grid_dep_launch_dependents()") > held, os.path.basename(path)


def test_bounds_sites_name_one_file():
    """A failed check reports DA_BOUNDS_FILE * 100000 + line: every file has a number of its own."""
    of = {}
    for path in HEADERS:
        for n in re.findall(r"#define DA_BOUNDS_FILE (\d+)", _code(path)):
            if n != "0":
                of.setdefault(int(n), []).append(os.path.basename(path))
    assert of and all(len(files) == 1 for files in of.values()), of
