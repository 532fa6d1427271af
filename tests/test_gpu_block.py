"""GPU parity of the block's operators against the fp64 oracle.

Bounds, per element:
  products    an instruction adds 16 exact products into the fp32 accumulator, aligned to the largest and cut
              off: two units in the last place (2^-23 each) of the sum S of the terms' magnitudes cover it, so a
              contraction of K is within (K / 16 + 2) 2^-22 S of z.  Activations have slopes up to 1.13 and are
              evaluated within 2^-19 (|z| + |act(z)|) (fast exponential: 2 ulp of a value and the rounding of
              its argument, up to 16 here).  Each bf16 rounding adds 2^-8 of the value, fp32 2^-24.
  gradients   dz rounded to bf16 adds 2^-8 of the sum of its terms' magnitudes; slopes are evaluated like
              the activations.
  norms       fp32 sums of D squares and the reciprocal root are within 2^-18 relative; a value combined from
              several terms within 2^-17 of the sum of their magnitudes; a sum over rows within
              (rows 2^-24 + 2^-17) of its terms' magnitudes.
"""

import numpy as np
import pytest
import torch

from differential_attention_03_gb300 import binding as da
from oracle import block

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from differential_attention_03_gb300 import build
    build.build()
    torch.cuda.init()


def _f64(t):
    return t.detach().double().cpu().numpy()


def _rnd(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape, std=1.0, dtype=BF):
        return (std * torch.randn(shape, generator=g, device="cuda")).to(dtype)
    return rnd


def _half(dtype):
    return 2.0 ** -8 if dtype == BF else 2.0 ** -24


def _within(got, ref, bound, what=""):
    got = _f64(got).reshape(ref.shape)
    over = np.abs(got - ref) - bound
    assert np.all(over <= 0), (what, float(np.max(over)), np.unravel_index(np.argmax(over), over.shape))


def _acc(K):
    return (K / 16 + 2) * 2.0 ** -22


def _check_linear(a, w, out, pre=None, bias=None, act="none", residual=None):
    K = a.shape[-1]
    A, W = _f64(a).reshape(-1, K), _f64(w)
    bias = None if bias is None else _f64(bias)
    res = None if residual is None else _f64(residual).reshape(-1, W.shape[0])
    ref, z = block.linear(A, W, bias, act, res)
    S = np.abs(A) @ np.abs(W).T + (0 if bias is None else np.abs(bias))
    ez = _acc(K) * S
    if pre is not None:
        _within(pre, z, ez + _half(BF) * np.abs(z) + 2.0 ** -8 * ez, "pre")
    v = block.activation(z, act)[0]
    e = 1.13 * ez + (0 if act == "none" else 2.0 ** -19 * (np.abs(z) + np.abs(v))) + (0 if res is None else 2.0 ** -24 * (np.abs(ref)))
    _within(out, ref, e + _half(out.dtype) * (np.abs(ref) + e) + 1e-37, "out")


@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (1, 2048, 1024), (3, 264, 72), (17, 128, 64), (64, 512, 1032), (130, 264, 200),
                                   (257, 776, 136), (300, 1032, 520), (1025, 256, 128), (513, 136, 2048)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_linear(M, N, K, dtype):
    rnd = _rnd(M + N + K)
    a, w = rnd(M, K), rnd(N, K, std=K ** -0.5)
    bias, res = rnd(N, dtype=F32), rnd(M, N, dtype=dtype)
    _check_linear(a, w, da.linear(a, w, dtype=dtype))
    _check_linear(a, w, da.linear(a, w, bias=bias, residual=res, dtype=dtype), bias=bias, residual=res)
    out, pre = da.linear_train(a, w, bias=bias, act="gelu", residual=res, dtype=dtype)
    da.device_status()
    _check_linear(a, w, out, pre, bias, "gelu", res)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [5, 200])
def test_linear_activations(act, M):
    rnd = _rnd(7)
    a, w, bias = rnd(M, 128), rnd(136, 128, std=0.3), rnd(136, dtype=F32)
    for dtype in (BF, F32):
        out, pre = da.linear_train(a, w, bias=bias, act=act, dtype=dtype)
        _check_linear(a, w, out, pre, bias, act)
    da.device_status()


@pytest.mark.parametrize("M", [2, 40, 300])
def test_linear_rows_apart_and_in_place(M):
    """Columns of wider tensors, and the residual stream updated in place."""
    rnd = _rnd(11)
    wide, w = rnd(M, 3 * 96), rnd(72, 96)
    a = wide[:, 96:192]
    for dtype in (BF, F32):
        out = torch.full((M, 4 * 72), 7.0, device="cuda", dtype=dtype)
        stream = rnd(M, 2 * 72, dtype=dtype)
        da.linear(a, w, residual=stream[:, 72:], out=out[:, 72:144])
        da.device_status()
        _check_linear(a, w, out[:, 72:144], residual=stream[:, 72:])
        assert bool((out[:, :72] == 7).all()) and bool((out[:, 144:] == 7).all())
        keep = out[:, 72:144].clone()
        same = stream[:, 72:]
        assert da.linear(a, w, residual=same, out=same) is same
        assert torch.equal(same, keep)
    x3 = rnd(2, M, 96)
    assert da.linear(x3, w).shape == (2, M, 72)
    _check_linear(x3, w, da.linear(x3, w))


def test_linear_long_contraction_in_fp32_stays_near():
    """fp32 results of a contraction of 8192 are within 1e-6 of the product (relative, in norm)."""
    rnd = _rnd(5)
    for M in (8, 256):
        a, w = rnd(M, 8192), rnd(512, 8192, std=2.0 ** -6)
        ref = a.double() @ w.double().T
        got = da.linear(a, w, dtype=F32).double()
        assert float((got - ref).norm() / ref.norm()) < 1e-6
    a, dy = rnd(8192, 256), rnd(8192, 264)
    got = da.linear_backward(a, rnd(264, 256), dy, da=False)["dw"].double()
    ref = dy.double().t() @ a.double()
    assert float((got - ref).norm() / ref.norm()) < 1e-6


def _check_linear_backward(a, w, dy, got, pre=None, act="none", bias=False):
    (M, K), N = a.shape, w.shape[0]
    A, W, DY = _f64(a), _f64(w), _f64(dy)
    Z = None if pre is None else _f64(pre)
    rda, rdw, rdb, dz = block.linear_backward(A, W, DY, Z, act)
    e = 0.0 if act == "none" else 2.0 ** -18 * np.abs(DY) * (1 + np.abs(Z)) + 2.0 ** -8 * np.abs(dz)
    eb = 0.0 if act == "none" else 2.0 ** -18 * np.abs(DY) * (1 + np.abs(Z))
    D = np.abs(dz) + e
    Da, Dw = D @ np.abs(W), D.T @ np.abs(A)
    ea = (e @ np.abs(W) if act != "none" else 0.0) + _acc(N) * Da
    ew = (e.T @ np.abs(A) if act != "none" else 0.0) + _acc(M) * Dw
    if "da" in got:
        _within(got["da"], rda, ea + _half(BF) * (np.abs(rda) + ea), "da")
    if "dw" in got:
        _within(got["dw"], rdw, ew + _half(got["dw"].dtype) * (np.abs(rdw) + ew), "dw")
    if bias:
        _within(got["dbias"], rdb, (eb.sum(0) if act != "none" else 0.0) + (M * 2.0 ** -24 + 2.0 ** -20) * np.abs(dz).sum(0), "dbias")


@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (3, 264, 72), (64, 512, 200), (130, 264, 1032), (1000, 136, 264), (257, 1048, 776),
                                   (2050, 64, 128)])
@pytest.mark.parametrize("act", ACTS)
def test_linear_backward(M, N, K, act):
    rnd = _rnd(M + 3 * N + K)
    a, w, dy, pre = rnd(M, K), rnd(N, K), rnd(M, N), rnd(M, N)
    for dt in (BF, F32):
        got = da.linear_backward(a, w, dy, pre=pre, act=act, bias=True, dw_dtype=dt)
        da.device_status()
        assert got["dw"].dtype == dt
        _check_linear_backward(a, w, dy, got, pre, act, True)
    again = da.linear_backward(a, w, dy, pre=pre, act=act, bias=True, dw_dtype=dt)
    for k in got:
        assert torch.equal(got[k], again[k]), k


def test_linear_backward_in_parts_and_rows_apart():
    rnd = _rnd(21)
    M, N, K = 77, 104, 88
    wa, wy, w, pre = rnd(M, 3 * K), rnd(M, 2 * N), rnd(N, K), rnd(M, N)
    a, dy = wa[:, K:2 * K], wy[:, N:]
    for act in ("none", "silu"):
        whole = da.linear_backward(a, w, dy, pre=pre, act=act, bias=True)
        _check_linear_backward(a, w, dy, whole, pre, act, True)
        for kw in (dict(dw=False), dict(da=False), dict(da=False, dw=False, bias=True), dict(bias=True, da=False)):
            part = da.linear_backward(a, w, dy, pre=pre, act=act, **kw)
            for k, t in part.items():
                assert torch.equal(t, whole[k]), (act, kw, k)
    da.device_status()


def test_backward_of_no_rows_is_zero():
    rnd = _rnd(22)
    w = rnd(16, 24)
    got = da.linear_backward(rnd(0, 24), w, rnd(0, 16), pre=rnd(0, 16), act="relu", bias=True)
    assert got["da"].shape == (0, 24) and not got["dw"].any() and not got["dbias"].any()
    got = da.gated_linear_backward(rnd(0, 24), w, rnd(0, 16), rnd(0, 8))
    assert got["dx"].shape == (0, 24) and not got["dw"].any()
    assert da.linear(rnd(0, 24), w).shape == (0, 16) and da.gated_linear(rnd(0, 24), w).shape == (0, 8)
    got = da.residual_norm_backward(rnd(0, 24), rnd(0, 24), rnd(0, 24), gamma_post=rnd(24, dtype=F32),
                                    gate=rnd(24, dtype=F32))
    assert not got["dgamma"].any() and not got["dgamma_post"].any() and not got["dgate"].any()
    y, s = da.residual_norm(rnd(0, 24))
    assert y.shape == s.shape == (0, 24)
    da.device_status()


def _check_gated(x, w, h, gu, act):
    K = x.shape[-1]
    X, W = _f64(x).reshape(-1, K), _f64(w)
    F = W.shape[0] // 2
    ref, rgu = block.gated_linear(X, W, act)
    e = _acc(K) * (np.abs(X) @ np.abs(W).T)
    if gu is not None:
        _within(gu, rgu, e + _half(BF) * (np.abs(rgu) + e), "gu")
    g, u, eg, eu = rgu[:, :F], rgu[:, F:], e[:, :F], e[:, F:]
    v = block.activation(g, act)[0]
    ev = 1.13 * eg + 2.0 ** -19 * (np.abs(g) + np.abs(v))
    eh = np.abs(u) * ev + np.abs(v) * eu + ev * eu
    _within(h, ref, eh + _half(BF) * (np.abs(ref) + eh), "h")


@pytest.mark.parametrize("M,D,F", [(1, 8, 8), (1, 1024, 2736), (5, 72, 136), (48, 264, 200), (130, 64, 264), (300, 520, 392),
                                   (1030, 128, 72)])
@pytest.mark.parametrize("act", ACTS)
def test_gated(M, D, F, act):
    rnd = _rnd(M + D + 5 * F)
    x, w = rnd(M, D), rnd(2 * F, D, std=D ** -0.5)
    h, gu = da.gated_linear_train(x, w, act=act)
    da.device_status()
    _check_gated(x, w, h, gu, act)
    assert torch.equal(da.gated_linear(x, w, act=act), h)


@pytest.mark.parametrize("M", [3, 200])
def test_gated_rows_apart(M):
    rnd = _rnd(31)
    wide, w = rnd(M, 256), rnd(2 * 40, 128, std=0.1)
    out = torch.full((M, 120), 3.0, device="cuda", dtype=BF)
    da.gated_linear(wide[:, 128:], w, out=out[:, 40:80])
    da.device_status()
    _check_gated(wide[:, 128:], w, out[:, 40:80], None, "silu")
    assert bool((out[:, :40] == 3).all()) and bool((out[:, 80:] == 3).all())


@pytest.mark.parametrize("M,D,F", [(1, 8, 8), (5, 72, 136), (130, 264, 72), (700, 136, 200), (257, 520, 264)])
@pytest.mark.parametrize("act", ACTS)
def test_gated_backward(M, D, F, act):
    rnd = _rnd(M + D + 7 * F)
    x, w, gu, dh = rnd(M, D), rnd(2 * F, D), rnd(M, 2 * F), rnd(M, F)
    for dt in (BF, F32):
        got = da.gated_linear_backward(x, w, gu, dh, act=act, dw_dtype=dt)
        da.device_status()
        X, W, GU, DH = _f64(x), _f64(w), _f64(gu), _f64(dh)
        rdx, rdw, dgu = block.gated_linear_backward(X, W, GU, DH, act)
        g, u = GU[:, :F], GU[:, F:]
        v = block.activation(g, act)[0]
        e = np.concatenate([2.0 ** -18 * np.abs(DH * u) * (1 + np.abs(g)), 2.0 ** -19 * np.abs(DH) * (np.abs(g) + np.abs(v))], 1)
        e += 2.0 ** -8 * np.abs(dgu)
        A = np.abs(dgu) + e
        ex = e @ np.abs(W) + _acc(2 * F) * (A @ np.abs(W))
        ew = e.T @ np.abs(X) + _acc(M) * (A.T @ np.abs(X))
        _within(got["dx"], rdx, ex + _half(BF) * (np.abs(rdx) + ex), "dx")
        _within(got["dw"], rdw, ew + _half(dt) * (np.abs(rdw) + ew), "dw")
        one = da.gated_linear_backward(x, w, gu, dh, act=act, dw=False)
        assert list(one) == ["dx"] and torch.equal(one["dx"], got["dx"])


TYPES = {"bf16": (BF, BF), "mixed": (BF, F32), "f32": (F32, F32)}


def _norm_inputs(rows, D, types, post, G, seed):
    dt, sdt = TYPES[types]
    rnd = _rnd(seed)
    x, res = rnd(rows, D, dtype=dt), rnd(rows, D, std=2.0, dtype=sdt)
    gate = 1 + rnd(G, D, std=0.3, dtype=F32) if G else None
    gp = 1 + rnd(D, std=0.2, dtype=F32) if post else None
    ga = 1 + rnd(D, std=0.2, dtype=F32)
    return x, res, gate, gp, ga, rnd(rows, D, dtype=dt), rnd(rows, D, dtype=sdt)


def _opt(t):
    return None if t is None else _f64(t)


def _check_norm(x, res, gate, gp, ga, scale, y, s):
    X, R, gate, gp = _f64(x), _opt(res), _opt(gate), _opt(gp)
    ry, rs = block.residual_norm(X, R, gate, scale, gp is not None, gp, _opt(ga))
    part = np.abs(rs - (0 if R is None else R))
    e = 2.0 ** -17 * (part + (0 if R is None else np.abs(R)))
    _within(s, rs, e + _half(s.dtype) * (np.abs(rs) + e) + 1e-37, "s")
    if y is not None:
        # y per s: y = s gamma / rms(s).  (Not |y| / |s|: where scale x cancels the residual exactly in 64 bits, as 0.7 * 10 - 7
        # does, that is 0, but scale is a float, and 0.7f * 10 - 7 = -1.2e-7, within e.)
        f = np.abs(1.0 if ga is None else _f64(ga)) / np.sqrt((rs * rs).mean(-1, keepdims=True) + 1e-5)
        ey = f * e + 2.0 ** -17 * np.abs(ry) + np.abs(ry) * np.sqrt((e * e).mean(-1, keepdims=True) / ((rs * rs).mean(-1, keepdims=True) + 1e-5))
        _within(y, ry, ey + _half(y.dtype) * (np.abs(ry) + ey) + 1e-37, "y")


NORM_SHAPES = [(1, 1, 0), (1, 8, 1), (6, 33, 2), (6, 64, 6), (30, 248, 3), (4, 257, 0), (7, 264, 7), (12, 1000, 3), (5, 2048, 5),
               (9, 4096, 1), (3, 4099, 3), (4, 8192, 2), (2, 8191, 1), (700, 128, 2), (1500, 512, 3)]


@pytest.mark.parametrize("rows,D,G", NORM_SHAPES)
@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("post", [False, True])
def test_norm(rows, D, G, types, post):
    x, res, gate, gp, ga, dy, ds = _norm_inputs(rows, D, types, post, G, rows + D)
    y, s = da.residual_norm(x, res, gate=gate, scale=0.7, gamma_post=gp, gamma=ga)
    da.device_status()
    assert y.dtype == x.dtype and s.dtype == res.dtype
    _check_norm(x, res, gate, gp, ga, 0.7, y, s)


@pytest.mark.parametrize("rows,D,G", NORM_SHAPES)
@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("post", [False, True])
def test_norm_backward(rows, D, G, types, post):
    x, res, gate, gp, ga, dy, ds = _norm_inputs(rows, D, types, post, G, rows + 2 * D)
    s = da.residual_norm(x, res, gate=gate, scale=0.7, gamma_post=gp, gamma=ga)[1]
    a = dict(gate=gate, scale=0.7, gamma_post=gp, gamma=ga)
    got = da.residual_norm_backward(x, s, dy, ds, **a)
    da.device_status()
    again = da.residual_norm_backward(x, s, dy, ds, **a)
    for k in got:
        assert torch.equal(got[k], again[k]), k
    _check_norm_backward(x, s, dy, ds, gate, gp, ga, 0.7, got)


def _check_norm_backward(x, s, dy, ds, gate, gp, ga, scale, got, post=None):
    X, S, DY, DS, gate, gp, ga = (_opt(t) for t in (x, s, dy, ds, gate, gp, ga))
    post = gp is not None if post is None else post
    rows = X.shape[0]
    ref = block.residual_norm_backward(X, S, DY, DS, gate, scale, post, gp, ga)
    assert set(got) == set(ref)
    rel = 2.0 ** -17
    rs = 1 / np.sqrt((S * S).mean(-1, keepdims=True) + 1e-5)
    T = np.zeros_like(X) if DS is None else np.abs(DS)
    if DY is not None:
        n, dn = S * rs, DY * (1.0 if ga is None else ga)
        T = T + rs * (np.abs(dn) + np.abs(n) * np.abs(dn * n).mean(-1, keepdims=True))
        _within(got["dgamma"], ref["dgamma"], (rows * 2.0 ** -24 + rel) * np.abs(DY * n).sum(0) + 1e-37, "dgamma")
    et = rel * T
    _within(got["dresidual"], ref["dresidual"], et + _half(s.dtype) * (np.abs(ref["dresidual"]) + et) + 1e-37, "dresidual")
    g = 1.0 if gate is None else np.repeat(gate.reshape(-1, X.shape[1]), rows // (gate.size // X.shape[1]), 0)
    DP = scale * np.abs(g) * T  # magnitudes behind dp
    if post:
        q = 1.0 if gp is None else gp
        rx = 1 / np.sqrt((X * X).mean(-1, keepdims=True) + 1e-5)
        xh = X * rx
        P = np.abs(xh * q)
        ex = 3 * rel * rx * (DP * np.abs(q) + np.abs(xh) * (DP * np.abs(q * xh)).mean(-1, keepdims=True))
        _within(got["dgamma_post"], ref["dgamma_post"], (rows * 2.0 ** -24 + 3 * rel) * (DP * np.abs(xh)).sum(0) + 1e-37, "dgamma_post")
    else:
        P, ex = np.abs(X), 2 * rel * DP
    _within(got["dx"], ref["dx"], ex + _half(x.dtype) * (np.abs(ref["dx"]) + ex) + 1e-37, "dx")
    if gate is not None:
        G = gate.size // X.shape[1]
        e = (rows * 2.0 ** -24 + 3 * rel) * (scale * T * P).reshape(G, rows // G, -1).sum(1)
        _within(got["dgate"], ref["dgate"], e + 1e-37, "dgate")


@pytest.mark.parametrize("rows,D,G", [(400, 4104, 4), (310, 5120, 155), (170, 6144, 1), (160, 8192, 80), (500, 4104, 500), (4000, 1000, 8),
                                      (2700, 1152, 0), (2000, 1001, 2), (900, 2050, 0)])
@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("post", [False, True])
def test_norm_more_rows_than_workers(rows, D, G, types, post):
    """Several rows a CTA, and of the backward pass several groups of rows."""
    x, res, gate, gp, ga, dy, ds = _norm_inputs(rows, D, types, post, G, rows + 3 * D)
    y, s = da.residual_norm(x, res, gate=gate, scale=0.7, gamma_post=gp, gamma=ga)
    _check_norm(x, res, gate, gp, ga, 0.7, y, s)
    got = da.residual_norm_backward(x, s, dy, ds, gate=gate, scale=0.7, gamma_post=gp, gamma=ga)
    da.device_status()
    _check_norm_backward(x, s, dy, ds, gate, gp, ga, 0.7, got)


@pytest.mark.parametrize("D", [72, 300, 1000])
def test_norm_parts(D):
    """Each part of the norms left out, and what may be written in place."""
    rnd = _rnd(D)
    rows = 10
    for dt, sdt in TYPES.values():
        x, res, dy, ds = rnd(rows, D, dtype=dt), rnd(rows, D, dtype=sdt), rnd(rows, D, dtype=dt), rnd(rows, D, dtype=sdt)
        y, s = da.residual_norm(x)  # a plain norm
        _check_norm(x, None, None, None, None, 1.0, y, s)
        y, s = da.residual_norm(x, res, norm=False)
        assert y is None
        _check_norm(x, res, None, None, None, 1.0, None, s)
        y, s = da.residual_norm(x, res, post=True)
        _check_norm(x, res, None, torch.ones(D, device="cuda"), None, 1.0, y, s)
        stream = res.clone()
        y2, s2 = da.residual_norm(x, stream, post=True, out=stream)
        assert s2 is stream and torch.equal(stream, s) and torch.equal(y2, y)
        assert da.residual_norm(x, stream_dtype=sdt)[1].dtype == sdt
        got = da.residual_norm_backward(x, s, dy, None, post=True)
        _check_norm_backward(x, s, dy, None, None, None, None, 1.0, got, True)
        got = da.residual_norm_backward(x, s, None, ds, scale=0.5)
        _check_norm_backward(x, s, None, ds, None, None, None, 0.5, got)
        kept = ds.clone()
        got = da.residual_norm_backward(x, s, dy, ds, scale=0.5)
        _check_norm_backward(x, s, dy, ds, None, None, None, 0.5, got)
        same = da.residual_norm_backward(x, s, dy, kept, scale=0.5, out={"dresidual": kept})
        assert same["dresidual"] is kept and torch.equal(kept, got["dresidual"]) and torch.equal(same["dx"], got["dx"])
    da.device_status()


def test_norm_gate_shapes():
    rnd = _rnd(3)
    B, n, D = 3, 5, 48
    x, res = rnd(B, n, D), rnd(B, n, D)
    for gate in (rnd(D, dtype=F32), rnd(B, D, dtype=F32), rnd(B, n, D, dtype=F32)):
        y, s = da.residual_norm(x, res, gate=gate, scale=0.3)
        g2 = gate.reshape(-1, D)
        _check_norm(x.view(-1, D), res.view(-1, D), g2, None, None, 0.3, y, s)
        got = da.residual_norm_backward(x, s, x, res, gate=gate, scale=0.3)
        assert got["dgate"].shape == gate.shape
        flat = {k: v.reshape(-1, D) if v.dim() > 1 else (v.reshape(1, D) if k == "dgate" else v) for k, v in got.items()}
        _check_norm_backward(x.view(-1, D), s.view(-1, D), x.view(-1, D), res.view(-1, D), g2, None, None, 0.3, flat)
    da.device_status()
