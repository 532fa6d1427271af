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


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("T", [1, 16])
def test_products_behind_a_tree_decode(T, fmt):
    """The attention of a serving step, W^O with the residual, the gated half, and the next step's attention behind it."""
    rnd = _rnd(T)
    B, n, H, d = 2, 640, 4, 64
    D = 2 * H * d
    cache = da.cache_v1(B, n, H, d, fmt)
    lens = torch.full((B,), 600, device="cuda", dtype=torch.int32)
    da.cache_append(cache, rnd(B, 600, H, d), rnd(B, 600, H, d), rnd(B, 600, H, 2 * d), lens=torch.zeros_like(lens))
    lam = torch.full((1,), 0.3, device="cuda")
    wo, wg, wd, wq = rnd(D, D, std=D ** -0.5), rnd(2 * 680, D, std=D ** -0.5), rnd(D, 680, std=680 ** -0.5), rnd(2 * H * d, D, std=D ** -0.5)
    q0, x0 = rnd(B, T, 2, H, d), rnd(B, T, D)

    def step(q, x, sync):
        outs = []

        def keep(t):
            outs.append(t)
            if sync:
                torch.cuda.synchronize()
            return t
        for _ in range(4):
            o = keep(da.tree_decode(q[:, :, 0].contiguous(), q[:, :, 1].contiguous(), cache, lam, 0.8, lens=lens))
            x = keep(da.linear(o.view(B, T, D), wo, residual=x))
            h = keep(da.gated_linear(x, wg))
            x = keep(da.linear(h, wd, residual=x))
            q = keep(da.linear(x, wq)).view(B, T, 2, H, d)
        return outs
    want = step(q0, x0, True)
    for _ in range(5):
        for i, (a, b) in enumerate(zip(step(q0, x0, False), want)):
            assert torch.equal(a, b), i
    da.device_status()


def test_two_streams_at_once():
    """Products for few tokens (clusters, tensor memory shared by two CTAs of an SM), tiles, norms and gradients of two streams
    beside each other: each gives what it gives alone."""
    sides = []
    for k, M in ((0, 24), (1, 130)):
        rnd = _rnd(k)
        D, F = 1024, 2056
        x, w, wg, wd, bias = rnd(M, D), rnd(D, D, std=D ** -0.5), rnd(2 * F, D, std=D ** -0.5), rnd(D, F, std=F ** -0.5), rnd(D, dtype=F32)
        big, wide = rnd(1300, D), rnd(2312, D, std=D ** -0.5)

        def work(s, x=x, w=w, wg=wg, wd=wd, bias=bias, big=big, wide=wide):
            y, r = da.residual_norm(x, stream=s)
            a = da.linear(y, w, bias=bias, act="gelu", residual=r, stream=s)
            f = da.linear(a, wide, dtype=F32, stream=s)
            h, gu = da.gated_linear_train(a, wg, stream=s)
            o = da.linear(h, wd, residual=a, stream=s)
            b = da.linear(big, wide, act="silu", stream=s)
            g = da.gated_linear_backward(a, wg, gu, h, stream=s)
            n = da.residual_norm_backward(x, r, o, a, stream=s)
            return [y, r, a, f, h, o, b, *g.values(), *n.values()]
        want = work(None)
        torch.cuda.synchronize()
        sides.append((torch.cuda.Stream(), work, want))
    outs = [[], []]
    for _ in range(30):
        for k, (s, work, _) in enumerate(sides):
            outs[k].append(work(s))
    torch.cuda.synchronize()
    for k, (_, _, want) in enumerate(sides):
        for got in outs[k]:
            for i, (p, q) in enumerate(zip(got, want)):
                assert torch.equal(p, q), (k, i)
    da.device_status()
