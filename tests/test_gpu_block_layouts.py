"""The products in every layout of their tiles, held to 64 bits: whole and half tiles, whole tiles with halves behind them,
on single SMs and on SM pairs, with every part of the epilogue.

Each case asserts the layout that its sizes get (a plan is made from estimates, so that sizes alone say little), and ends
inside a tile in both directions.  The bounds are those of test_gpu_block.py: (K / 16 + 2) 2^-22 of the sum of the terms'
magnitudes for a product, 2^-19 (|z| + |act(z)|) for an activation, half a step for each rounding.
"""

import math

import pytest
import torch

from differential_attention_03_gb300 import binding as da

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
BF, F32 = torch.bfloat16, torch.float32
# (SMs of a cluster, whole tiles, tiles in halves) and sizes that get them: M, N, K of the product
LINEAR = [((1, False, True), (133, 4104, 72)), ((2, False, True), (1030, 1288, 4104)), ((1, True, False), (1030, 2312, 520)),
          ((2, True, False), (771, 4104, 2056)), ((1, True, True), (2051, 2056, 520)), ((2, True, True), (2051, 2056, 1032))]
GATED = [((1, False, True), (131, 2056, 72)), ((2, False, True), (131, 2568, 4104)), ((1, True, False), (261, 4104, 520)),
         ((2, True, False), (261, 4104, 2056)), ((1, True, True), (1030, 2056, 520)), ((2, True, True), (1030, 2056, 1032))]
# ... M, N, K of the call whose da or dw it is
DA = [((1, False, True), (131, 72, 136)), ((2, False, True), (131, 4104, 2568)), ((1, True, False), (1032, 520, 2056)),
      ((2, True, False), (1029, 2056, 2056)), ((1, True, True), (2051, 520, 2056)), ((2, True, True), (2051, 1032, 2056))]
DW = [((1, False, True), (131, 72, 136)), ((2, False, True), (4101, 136, 264)), ((1, True, False), (1030, 2056, 1032)),
      ((2, True, False), (2051, 1032, 2056)), ((1, True, True), (520, 2056, 2056)), ((2, True, True), (1029, 2056, 2056))]


def _names(cases):
    return ["{}-{}{}".format("x".join(map(str, s)), "pairs" if k[0] == 2 else "single",
                             "-whole-half" if k[1] and k[2] else "-whole" if k[1] else "-half") for k, s in cases]


def _over(kind, cases):
    return pytest.mark.parametrize("layout,sizes", cases, ids=_names(cases))


@pytest.fixture(scope="module", autouse=True)
def _built():
    from differential_attention_03_gb300 import build
    build.build()
    torch.cuda.init()


def _runs_as(layout, kind, M, N, K):
    p = da.debug_product_plan(kind, M, N, K)
    assert p["kernel"] == "tiles" and (p["cluster"], p["whole"] > 0, p["halved"] > 0) == layout, p


def _rnd(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape, std=1.0, dtype=BF):
        return (std * torch.randn(shape, generator=g, device="cuda")).to(dtype)
    return rnd


def _half(dtype):
    return 2.0 ** -8 if dtype == BF else 2.0 ** -24


def _acc(K):
    return (K / 16 + 2) * 2.0 ** -22


def _within(got, ref, bound, what):
    over = (got.double() - ref).abs() - bound
    assert bool((over <= 0).all()), (what, float(over.max()), divmod(int(over.argmax()), ref.shape[-1]))


def _value(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z) if act == "silu" else z


class Product:
    """a w^T in 64 bits, and how far off a kernel's may be."""

    def __init__(self, a, w):
        A, W = a.double(), w.double()
        self.z = A @ W.T
        self.S = A.abs() @ W.abs().T
        self.acc = _acc(a.shape[1])

    def check(self, out, pre=None, bias=None, act="none", residual=None):
        z = self.z if bias is None else self.z + bias.double()
        ez = self.acc * (self.S if bias is None else self.S + bias.double().abs())
        if pre is not None:
            _within(pre, z, ez + _half(BF) * (z.abs() + ez), "pre")
        v = _value(z, act)
        ref = v if residual is None else v + residual.double()
        e = 1.13 * ez + (0 if act == "none" else 2.0 ** -19 * (z.abs() + v.abs())) + 2.0 ** -24 * ref.abs()
        _within(out, ref, e + _half(out.dtype) * (ref.abs() + e) + 1e-37, act)


@pytest.mark.parametrize("dtype", [BF, F32])
@_over("linear", LINEAR)
def test_linear_layouts(layout, sizes, dtype):
    """Nothing but the product, every part of the epilogue alone, and all of them with the residual updated in place."""
    M, N, K = sizes
    _runs_as(layout, "linear", M, N, K)
    rnd = _rnd(M + N + K)
    wide = torch.full((M, K + 64), float("nan"), device="cuda", dtype=BF)  # (columns of a wider tensor)
    a, w = wide[:, 32:32 + K], rnd(N, K, std=K ** -0.5)
    a.copy_(rnd(M, K))
    bias, res = rnd(N, dtype=F32), rnd(M, N, dtype=dtype)
    ref = Product(a, w)
    ref.check(da.linear(a, w, dtype=dtype))
    ref.check(da.linear(a, w, bias=bias, dtype=dtype), bias=bias)
    ref.check(da.linear(a, w, residual=res, dtype=dtype), residual=res)
    out, pre = da.linear_train(a, w, dtype=dtype)
    ref.check(out, pre)
    out, pre = da.linear_train(a, w, bias=bias, act="gelu", residual=res, dtype=dtype)
    ref.check(out, pre, bias, "gelu", res)
    stream = torch.full((M + 2, N + 64), 7.0, device="cuda", dtype=dtype)
    same = stream[1:M + 1, 32:32 + N]
    same.copy_(res)
    again, z = da.linear_train(a, w, bias=bias, act="gelu", residual=same, out=same)
    assert again is same and torch.equal(same, out) and torch.equal(z, pre)
    same.fill_(7)
    assert bool((stream == 7).all())
    da.device_status()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("which", [0, 5])
def test_linear_activations_in_tiles(act, which):
    layout, (M, N, K) = LINEAR[which]
    _runs_as(layout, "linear", M, N, K)
    rnd = _rnd(7)
    a, w, bias = rnd(M, K), rnd(N, K, std=2 * K ** -0.5), rnd(N, dtype=F32)
    ref = Product(a, w)
    for dtype in (BF, F32):
        out, pre = da.linear_train(a, w, bias=bias, act=act, dtype=dtype)
        ref.check(out, pre, bias, act)
        assert torch.equal(da.linear(a, w, bias=bias, act=act, dtype=dtype), out)
    da.device_status()


@pytest.mark.parametrize("act", ACTS)
@_over("gated", GATED)
def test_gated_layouts(layout, sizes, act):
    M, F, D = sizes
    _runs_as(layout, "gated", M, F, D)
    rnd = _rnd(M + F + D)
    x, w = rnd(M, D), rnd(2 * F, D, std=D ** -0.5)
    h, gu = da.gated_linear_train(x, w, act=act)
    X, W = x.double(), w.double()
    ref, e = X @ W.T, _acc(D) * (X.abs() @ W.abs().T)
    _within(gu, ref, e + _half(BF) * (ref.abs() + e), "gu")
    g, u, eg, eu = ref[:, :F], ref[:, F:], e[:, :F], e[:, F:]
    v = _value(g, act)
    ev = 1.13 * eg + 2.0 ** -19 * (g.abs() + v.abs())
    eh = u.abs() * ev + v.abs() * eu + ev * eu
    _within(h, v * u, eh + _half(BF) * ((v * u).abs() + eh), "h")
    wide = torch.full((M + 2, F + 64), 7.0, device="cuda", dtype=BF)
    out = wide[1:M + 1, 32:32 + F]
    assert torch.equal(da.gated_linear(x, w, act=act, out=out), h)
    out.fill_(7)
    assert bool((wide == 7).all())
    da.device_status()


@_over("da", DA)
def test_input_gradient_layouts(layout, sizes):
    M, N, K = sizes
    _runs_as(layout, "da", M, K, N)
    rnd = _rnd(M + N + K)
    w, dy = rnd(N, K), rnd(M, N)
    got = da.linear_backward(rnd(M, K), w, dy, dw=False)["da"]
    ref, e = dy.double() @ w.double(), _acc(N) * (dy.double().abs() @ w.double().abs())
    _within(got, ref, e + _half(BF) * (ref.abs() + e), "da")
    da.device_status()


@pytest.mark.parametrize("dtype", [BF, F32])
@_over("dw", DW)
def test_weight_gradient_layouts(layout, sizes, dtype):
    M, N, K = sizes
    _runs_as(layout, "dw", N, K, M)
    rnd = _rnd(M + N + K)
    a, dy = rnd(M, K), rnd(M, N)
    pool = torch.full((N + 2, K), 7.0, device="cuda", dtype=dtype)
    got = da.linear_backward(a, rnd(N, K), dy, da=False, dw_dtype=dtype, out={"dw": pool[1:N + 1]})["dw"]
    ref, e = dy.double().T @ a.double(), _acc(M) * (dy.double().abs().T @ a.double().abs())
    _within(got, ref, e + _half(dtype) * (ref.abs() + e), "dw")
    assert bool((pool[0] == 7).all()) and bool((pool[N + 1] == 7).all())
    da.device_status()
