"""fp32 outputs of long contractions: 512 values of K in an accumulator at most, in every form of the kernel for few tokens
(segments in accumulators of their own; taking turns in two, or in one; alone or in clusters) and in the tiles.

Positive terms, per element.  An instruction adds 16 products and cuts off at most two units in the last place (2^-23 each)
of the sum so far, which after j of a segment's 32 instructions is j / 32 of it: 2 * 2^-23 * 16.5 = 3.9e-6 of a segment.
n = K / 512 segments are added to nearest, 2^-24 of the sum so far each: 2^-24 (n + 1) / 2, 2.0e-6 for the longest here (32768).
(With all of K in one accumulator 8192 values are off by 3e-5, 4096 by 1.1e-5.)
Terms of both signs, in norm: 1e-6, the accuracy that fp32 products are documented with.
"""

import pytest
import torch

from differential_attention_03_gb300 import binding as da
from .test_gpu_block import _check_linear

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from differential_attention_03_gb300 import build
    build.build()
    torch.cuda.init()


@pytest.mark.parametrize("M,N,K", [(1, 8192, 8192), (48, 8192, 8192), (256, 8192, 8192), (1, 32768, 8192), (48, 32768, 8192),
                                   (256, 32768, 4096), (1, 8192, 16384), (48, 4096, 16384), (256, 4096, 16384), (130, 4096, 4096),
                                   (3, 1000, 32768), (128, 520, 32760), (17, 5000, 7000), (77, 2056, 12296)])
def test_long_contractions(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    a, w = (torch.rand(s, generator=g, device="cuda").to(BF) for s in ((M, K), (N, K)))
    got, ref = da.linear(a, w, dtype=F32).double(), a.double() @ w.double().T
    n = (K + 511) // 512
    assert float(((got - ref).abs() / ref).max()) < 2 * 2.0 ** -23 * 16.5 + 2.0 ** -24 * (n + 1) / 2
    a, w = (torch.randn(s, generator=g, device="cuda").to(BF) for s in ((M, K), (N, K)))
    got, ref = da.linear(a, w, dtype=F32), a.double() @ w.double().T
    assert float((got.double() - ref).norm() / ref.norm()) < 1e-6
    assert torch.equal(got, da.linear(a, w, dtype=F32))
    da.device_status()


@pytest.mark.parametrize("M,N,K", [(1, 8192, 8192), (40, 2048, 16392), (129, 4096, 4096), (128, 264, 32768), (5, 10928, 4104)])
def test_the_epilogue_behind_long_contractions(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(K)

    def rnd(*shape, std=1.0, dtype=BF):
        return (std * torch.randn(shape, generator=g, device="cuda")).to(dtype)
    a, w, bias, res = rnd(M, K), rnd(N, K, std=K ** -0.5), rnd(N, dtype=F32), rnd(M, N, dtype=F32)
    out, pre = da.linear_train(a, w, bias=bias, act="silu", residual=res, dtype=F32)
    da.device_status()
    _check_linear(a, w, out, pre, bias, "silu", res)
    _check_linear(a, w, da.linear(a, w, dtype=F32))
