"""The longest contraction of a product: a weight gradient over more rows than one wait's limit (2e9 cycles) is long.

A K block of 64 rows takes 270 cycles and more, and the epilogue of a bf16 output waits for all of them at once: 500 million rows
are 7.8 million blocks, 2.1e9 cycles at least (1.8 s were measured).  The limit of that wait grows with the blocks, so the call ends with its result,
not with ERR_TIMEOUT.  The rows are zeros but for a few, so that the result is known exactly.
"""

import pytest
import torch

from differential_attention_03_gb300 import binding as da

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from differential_attention_03_gb300 import build
    build.build()
    torch.cuda.init()


def test_a_weight_gradient_over_500_million_rows():
    M, N, K = 500_000_000, 8, 8
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    a, dy = torch.zeros(M, K, device="cuda", dtype=BF), torch.zeros(M, N, device="cuda", dtype=BF)
    g = torch.Generator(device="cuda").manual_seed(0)
    rows = torch.tensor([0, 63, 64, 123_456_789, 268_435_455, 268_435_456, 499_999_999], device="cuda")  # 2^28 rows are 2^31 values
    a[rows] = torch.randint(-3, 4, (len(rows), K), generator=g, device="cuda").to(BF)
    dy[rows] = torch.randint(-3, 4, (len(rows), N), generator=g, device="cuda").to(BF)
    want = dy[rows].double().T @ a[rows].double()
    w = torch.zeros(N, K, device="cuda", dtype=BF)
    for dtype in (BF, torch.float32):
        got = da.linear_backward(a, w, dy, da=False, dw_dtype=dtype)["dw"]
        assert torch.equal(got.double(), want), dtype
    da.device_status()
    del a, dy
    torch.cuda.empty_cache()
