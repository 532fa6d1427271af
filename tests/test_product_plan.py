"""Which kernel and layout a product's sizes get (host only)."""

import pytest

from differential_attention_03_gb300 import binding as da
from differential_attention_03_gb300 import build
from .test_gpu_block_layouts import DA, DW, GATED, LINEAR


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _layout(kind, M, N, K):
    p = da.debug_product_plan(kind, M, N, K)
    return (p["cluster"], p["whole"] > 0, p["halved"] > 0) if p["kernel"] == "tiles" else p["kernel"]


def test_the_layouts_tests_reach_every_layout():
    every = {(cluster, whole, halved) for cluster in (1, 2) for whole, halved in ((False, True), (True, False), (True, True))}
    for kind, cases in (("linear", LINEAR), ("gated", GATED)):
        assert {k for k, _ in cases} == every
        for layout, sizes in cases:
            assert _layout(kind, *sizes) == layout, (kind, sizes)
    assert {k for k, _ in DA} == every and {k for k, _ in DW} == every
    for layout, (M, N, K) in DA:
        assert _layout("da", M, K, N) == layout, (M, N, K)
    for layout, (M, N, K) in DW:
        assert _layout("dw", N, K, M) == layout, (M, N, K)


def test_few_tokens_get_their_kernel():
    for M in (1, 16, 48, 128):
        for kind in ("linear", "gated", "da"):
            assert _layout(kind, M, 2048, 2048) == "few"
        assert _layout("dw", 2048, 2048, M) != "few"


def test_bad_sizes_have_no_plan():
    for sizes in ((0, 8, 8), (8, 0, 8), (8, 8, 0), (-1, 8, 8)):
        with pytest.raises(ValueError):
            da.debug_product_plan("linear", *sizes)


def test_fp32_outputs_sum_512_values_in_an_accumulator():
    """The tensor cores cut off as they add: 1e-9 relative a value, whatever the kernel and its layout."""
    for M in (1, 2, 16, 17, 48, 100, 128, 129, 200, 256, 300, 512, 777, 2050):
        for N in (8, 72, 512, 1000, 2048, 4096, 8192, 32768, 128256):
            for K in (8, 72, 512, 520, 1000, 2048, 4096, 5472, 8192, 16384, 32768, 65536, 1048576):
                p = da.debug_product_plan("linear", M, N, K, f32=True)
                assert p["segment"] <= 512, (M, N, K, p)
                if p["kernel"] == "few":
                    assert p["width"] <= 256 and p["stages"] >= 1
    assert da.debug_product_plan("dw", 264, 256, 8192, f32=True)["segment"] <= 512
    assert da.debug_product_plan("linear", 1, 2048, 8192)["segment"] > 512  # (a bf16 output does not see it)
