"""Calls whose inputs the kernel just before them writes: the products are programmatic dependents, whose CTAs are up while
that kernel still runs, and read nothing before its end."""

import pytest
import torch

from differential_attention_03_gb300 import binding as da

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from differential_attention_03_gb300 import build
    build.build()
    torch.cuda.init()


def _rnd(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape, std=1.0, dtype=BF):
        return (std * torch.randn(shape, generator=g, device="cuda")).to(dtype)
    return rnd


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K", [(1, 4096, 256), (3, 264, 72), (300, 4096, 256), (1030, 2312, 520), (2051, 2056, 1032)])
def test_a_bias_of_the_product_before(M, N, K, dtype):
    """A bias that depends on a condition: an fp32 row of one product, the bias of the next, over and over."""
    rnd = _rnd(N + K)
    a, w, wc = rnd(M, K), rnd(N, K, std=K ** -0.5), rnd(N, K)
    conditions = [rnd(1, K) for _ in range(3)]
    want = []
    for c in conditions:
        row = da.linear(c, wc, dtype=F32)[0].clone()
        torch.cuda.synchronize()
        want.append(da.linear(a, w, bias=row, dtype=dtype))
    row = torch.zeros(1, N, device="cuda", dtype=F32)
    outs = []
    for i in range(24):
        da.linear(conditions[i % 3], wc, out=row)
        outs.append(da.linear(a, w, bias=row[0], dtype=dtype))
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i % 3]), i
    da.device_status()


@pytest.mark.parametrize("M", [1, 40, 300, 2051])
def test_weights_rows_and_residuals_of_the_product_before(M):
    """Each operand in turn is what the kernel before wrote into a tensor that is used again."""
    rnd = _rnd(M)
    N, K = 2056, 520
    a0, w, w2 = rnd(M, N, std=0.1), rnd(N, K, std=K ** -0.5), rnd(N, N, std=N ** -0.5)
    xs = [rnd(M, K) for _ in range(3)]
    ws = [rnd(N, K, std=K ** -0.5) for _ in range(3)]
    h, y = torch.empty(M, N, device="cuda", dtype=BF), None
    eye = torch.eye(K, device="cuda", dtype=BF)
    made = torch.empty(N, K, device="cuda", dtype=BF)
    want, got = [], []
    for turn, out in ((0, want), (1, got)):
        for i in range(12):
            da.linear(xs[i % 3], w, act="silu", out=h)  # rows
            if not turn:
                torch.cuda.synchronize()
            y = da.linear(h, w2, residual=a0)
            if not turn:
                torch.cuda.synchronize()
            da.linear(ws[i % 3], eye, out=made)  # weights
            if not turn:
                torch.cuda.synchronize()
            z = da.linear(xs[(i + 1) % 3], made, residual=y)  # the residual and the weights
            if not turn:
                torch.cuda.synchronize()
            n, s = da.residual_norm(z, y)
            out.append((y, z, n, s))
    for i, (one, two) in enumerate(zip(want, got)):
        for p, q in zip(one, two):
            assert torch.equal(p, q), i
    da.device_status()
