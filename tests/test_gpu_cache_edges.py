"""Tree decode where the softmax is uneven: a key far above many equal ones, in units enough that one
partial state covers tens of thousands of keys.

Bar: a weight over an 8-bit cache stands in three e5m2 terms, within 2^-8.8 of itself or 2^-28 of the
largest contribution; the query's two terms, exp2 and the fp32 sums take another 2^-10: a map's output
is within E = (2^-8 + 2^-10) sum_j p_j |v_j|, whatever the number of keys (n 2^-28 of the largest
contribution is below 2^-11 of the sum for n up to 2^17).  The norm multiplies E by its gain and adds
the change of the row's rms; the output rounds to bf16.
"""

import copy
import math

import numpy as np
import pytest
import torch

import oracle
from differential_attention_03_gb300 import binding as da

pytestmark = pytest.mark.gpu

E_MAP = 2.0 ** -8 + 2.0 ** -10


@pytest.fixture(scope="module", autouse=True)
def _built():
    from differential_attention_03_gb300 import build
    build.build()
    torch.cuda.init()


def _np(t):
    return t.detach().float().cpu().double().numpy()


def _bf(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def _rows(codes, scales, x):
    """x as e4m3 rows with a scale each, written to the cache; the values they stand for."""
    s = x.abs().amax(-1) / 448.0
    codes.copy_((x / torch.where(s > 0, s, 1.0).unsqueeze(-1)).clamp(-448, 448))
    scales.copy_(s.transpose(1, 2))
    return _np(codes) * _np(s)[..., None]


def _fill(t, scales, scale, x, fmt):
    if fmt == "fp8":
        return _rows(t, scales, x)
    if fmt == "fp8k" and scale is not None:
        t.copy_((x / scale).clamp(-448, 448))
        return _np(t) * scale
    t.copy_(x)
    return _np(t)


def _uneven(q, n, sinks, nats):
    """Keys [1, n, 1, d] without a score, but for the sinks, which the first query row sees `nats` above."""
    d = q.shape[-1]
    k = torch.zeros((1, n, 1, d), device="cuda")
    along = q[:, 0].float()
    k[:, sinks] = (along * (nats * math.sqrt(d)) / along.square().sum(-1, keepdim=True)).unsqueeze(1)
    return k


def _values(g, n, dv, sinks):
    """Rows of mean 1 and spread 1; an ordinary row on the sinks, of the opposite sign."""
    v = 1.0 + torch.randn((1, n, 1, dv), generator=g, device="cuda")
    v[:, sinks] -= 2.0
    return v


def _everywhere(small, big):
    """A cache's contents for all sequences and heads of a larger one: enough units that a partial state
    covers tens of thousands of keys (the tiles of one head alone would be dealt out to all SMs)."""
    for name in ("k1", "k2", "v", "k1_scales", "k2_scales", "v_scales"):
        x, y = getattr(small, name), getattr(big, name)
        if x is not None:
            y.copy_(x.expand(y.shape))


@pytest.mark.parametrize("d,T", [(64, 1), (64, 7), (128, 14), (64, 20), (128, 27), (64, 64), (128, 40)])
@pytest.mark.parametrize("fmt,nats", [("fp8", 10.0), ("fp8", 11.5), ("fp8", 12.0), ("fp8", 13.0), ("fp8k", 12.0),
                                      ("bf16", 12.0)])
def test_small_weights_add_up_v1(d, T, fmt, nats):
    B, H, n, sinks = 4, 2048 // d, 32768, [130]
    g = torch.Generator(device="cuda").manual_seed(T)
    one, c = (da.cache_v1(b, n, h, d, fmt, k1_scale=0.06, k2_scale=0.06) for b, h in ((1, 1), (B, H)))
    q1, q2 = _bf(g, 1, T, 1, d), _bf(g, 1, T, 1, d)
    q1[:], q2[:] = q1[:, :1], q2[:, :1]  # (every token sees the sink as far above)
    k1 = _fill(one.k1, one.k1_scales, one.k1_scale, _uneven(q1, n, sinks, nats), fmt)
    k2 = _fill(one.k2, one.k2_scales, one.k2_scale, _uneven(q2, n, [n // 2], 3.0), fmt)
    v = _fill(one.v, one.v_scales, None, _values(g, n, 2 * d, sinks), fmt)
    _everywhere(one, c)
    lam = torch.tensor([0.25], device="cuda")
    out = da.tree_decode(q1.expand(B, T, H, d).contiguous(), q2.expand(B, T, H, d).contiguous(), c, lam, 0.2)
    da.device_status()
    ref, pre, spread, _, gain = oracle.tree_v1(q1.cpu(), q2.cpu(), k1, k2, v, [n - T], [T], None, 0.25, 0.2, np.ones(2 * d),
                                               1e-5)
    e = E_MAP * spread
    rms = np.sqrt((pre ** 2).mean(-1, keepdims=True) + 1e-5)
    de = np.sqrt((e ** 2).mean(-1, keepdims=True))
    bound = gain * (e + np.abs(pre) * de / np.maximum(rms - de, 1e-9))
    over = np.abs(_np(out) - ref) - (bound + 2.0 ** -8 * (np.abs(ref) + bound))
    assert over.max() <= 0, over.max()


@pytest.mark.parametrize("nats", [12.0, 13.0])
@pytest.mark.parametrize("T,pairs", [(1, 1), (6, 4), (20, 1), (33, 2)])
def test_small_weights_add_up_v2(T, pairs, nats):
    B, H, d, n, sinks = 4, 16, 128, 65536, [70, 40000]
    g = torch.Generator(device="cuda").manual_seed(pairs)
    one, c = da.cache_v2(1, n, 1, d, "fp8"), da.cache_v2(B, n, H, d, "fp8")
    q = _bf(g, 1, T, 1, d).expand(1, T, 2 * pairs, d).contiguous()
    q[:] = q[:, :1]
    q[:, :, 1::2] *= 0.25  # (the second map of each pair is nearly even)
    k = _rows(one.k1, one.k1_scales, _uneven(q[:, :, :1], n, sinks, nats))
    v = _rows(one.v, one.v_scales, _values(g, n, d, sinks))
    _everywhere(one, c)
    logits = torch.randn(pairs, generator=g, device="cuda")
    out = da.v2_tree_decode(q.repeat(B, 1, H, 1), c, logits.repeat(H))
    da.device_status()
    ref, spread, _ = oracle.tree_v2(q.cpu(), k, v, np.broadcast_to(_np(logits), (1, T, pairs)), [n - T], [T], None)
    ref, spread = np.tile(ref, (1, 1, H, 1)), np.tile(spread, (1, 1, H, 1))
    e = E_MAP * spread
    over = np.abs(_np(out) - ref) - (e + 2.0 ** -8 * (np.abs(ref) + e))
    assert over.max() <= 0, over.max()


@pytest.mark.parametrize("T", [1, 16, 24, 64])
def test_references_move_and_values_differ_in_size(T):
    # Scores that climb by 40 powers of e along the cache while the value rows shrink and grow by 2^40.
    H, d, n = 2, 64, 5000
    g = torch.Generator(device="cuda").manual_seed(T)
    c = da.cache_v1(1, n, H, d, "fp8")
    q1, q2 = _bf(g, 1, T, H, d), _bf(g, 1, T, H, d)
    q1[:], q2[:] = q1[:, :1], q2[:, :1]
    climb = torch.linspace(0, 40, n, device="cuda").view(1, n, 1, 1)
    keys = []
    for q, t, s, up in ((q1, c.k1, c.k1_scales, climb), (q2, c.k2, c.k2_scales, climb.flip(1))):
        along = q[:, :1].float()
        keys.append(_rows(t, s, along * (up * math.sqrt(d)) / along.square().sum(-1, keepdim=True)))
    size = torch.exp2(20 * torch.sin(torch.arange(n, device="cuda") / 300.0)).view(1, n, 1, 1)
    v = _rows(c.v, c.v_scales, (1.0 + torch.randn((1, n, H, 2 * d), generator=g, device="cuda")) * size)
    out = da.tree_decode(q1, q2, c, torch.tensor([0.25], device="cuda"), 0.2)
    da.device_status()
    ref, pre, spread, _, gain = oracle.tree_v1(q1.cpu(), q2.cpu(), *keys, v, [n - T], [T], None, 0.25, 0.2,
                                               np.ones(2 * d), 1e-5)
    # (scores of up to 40: fp32's sums of 64 products are off by 2^-24 of 64 such terms)
    e = (E_MAP + 40 * 64 * 2.0 ** -24) * spread
    rms = np.sqrt((pre ** 2).mean(-1, keepdims=True) + 1e-5)
    de = np.sqrt((e ** 2).mean(-1, keepdims=True))
    bound = gain * (e + np.abs(pre) * de / np.maximum(rms - de, 1e-9))
    over = np.abs(_np(out) - ref) - (bound + 2.0 ** -8 * (np.abs(ref) + bound))
    assert over.max() <= 0, over.max()


def _random(g, B, n, H, d, v1, fmt, k_mult=1.0):
    """A cache of random rows and the values they stand for: (cache, keys, values)."""
    dv, ks = (2 * d, (0.013 * k_mult, 0.021 * k_mult)) if v1 else (d, (0.013 * k_mult,))
    c = (da.cache_v1(B, n, H, d, fmt, k1_scale=ks[0], k2_scale=ks[1]) if v1 else
         da.cache_v2(B, n, H, d, fmt, k_scale=ks[0]))
    keys = [_fill(t, s, f, torch.randn((B, n, H, d), generator=g, device="cuda") * k_mult, fmt)
            for t, s, f in ((c.k1, c.k1_scales, c.k1_scale), (c.k2, c.k2_scales, c.k2_scale)) if t is not None]
    val = _fill(c.v, c.v_scales, None, torch.randn((B, n, H, dv), generator=g, device="cuda"), fmt)
    return c, keys, val


@pytest.mark.parametrize("fmt", ["bf16", "fp8k", "fp8"])
@pytest.mark.parametrize("v1,T,d", [(True, 1, 64), (True, 5, 64), (True, 14, 128), (True, 20, 64), (True, 40, 128),
                                    (False, 3, 128), (False, 30, 128)])
def test_non_finite_queries_give_nan(v1, T, d, fmt):
    B, H, n = 2, 2, 300
    g = torch.Generator(device="cuda").manual_seed(T + d)
    c, _, _ = _random(g, B, n, H, d, v1, fmt)
    q = [_bf(g, B, T, H if v1 else 4 * H, d) for _ in range(2)]
    lam, logits = torch.tensor([0.4], device="cuda"), torch.randn(2 * H, generator=g, device="cuda")
    lens = torch.tensor([n - T, 17], dtype=torch.int32, device="cuda")

    def call():
        out = da.tree_decode(*q, c, lam, 0.2, lens=lens) if v1 else da.v2_tree_decode(q[0], c, logits, lens=lens)
        da.device_status()
        return out
    clean = call()
    assert torch.isfinite(clean).all()
    want = torch.zeros(clean.shape[:3], dtype=torch.bool, device="cuda")
    for b, t, h, x in ((0, 0, 1, float("inf")), (1, T - 1, 0, float("-inf")), (1, T // 2, 1, float("nan"))):
        q[0][b, t, h, 3] = x
        want[b, t, h if v1 else h // 2] = True
    out = call()
    assert torch.equal(out.isnan().all(-1), want) and torch.equal(out.isnan().any(-1), want)
    # (the others' query rows may be scaled by another power of two: a rounding of the output apart)
    assert ((out - clean).abs() <= 2.0 ** -7 * clean.abs() + 2.0 ** -10)[~want].all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8k", "fp8"])
@pytest.mark.parametrize("T,d", [(2, 64), (20, 64), (40, 128)])
def test_large_queries_meet_small_keys(T, d, fmt):
    B, H, n, big = 1, 2, 200, 2.0 ** 115
    g = torch.Generator(device="cuda").manual_seed(T)
    c, keys, val = _random(g, B, n, H, d, True, fmt, 1 / big)
    q1, q2 = ((_bf(g, B, T, H, d).float() * big).to(torch.bfloat16) for _ in range(2))
    out = da.tree_decode(q1, q2, c, torch.tensor([0.37], device="cuda"), 0.3)
    da.device_status()
    ref, pre, spread, _, gain = oracle.tree_v1(q1.cpu(), q2.cpu(), *keys, val, [n - T], [T], None, float(np.float32(0.37)),
                                               0.3, np.ones(2 * d), 1e-5)
    e = E_MAP * spread
    rms = np.sqrt((pre ** 2).mean(-1, keepdims=True) + 1e-5)
    de = np.sqrt((e ** 2).mean(-1, keepdims=True))
    bound = gain * (e + np.abs(pre) * de / np.maximum(rms - de, 1e-9))
    over = np.abs(_np(out) - ref) - (bound + 2.0 ** -8 * (np.abs(ref) + bound))
    assert over.max() <= 0, over.max()


@pytest.mark.parametrize("fmt", ["bf16", "fp8k", "fp8"])
@pytest.mark.parametrize("T,d", [(3, 64), (20, 128), (40, 64)])
def test_scores_that_underflow_weigh_alike(T, d, fmt):
    # queries and keys of some 2^-100: every seen key weighs the same, a hidden one nothing
    B, H, n, tiny = 1, 2, 200, 2.0 ** -100
    g = torch.Generator(device="cuda").manual_seed(T)
    c, _, val = _random(g, B, n, H, d, True, fmt, tiny)
    q1, q2 = ((_bf(g, B, T, H, d).float() * tiny).to(torch.bfloat16) for _ in range(2))
    out = da.tree_decode(q1, q2, c, torch.tensor([0.25], device="cuda"), 0.0)
    da.device_status()
    for t in range(T):
        mean, size = val[0, :n - T + t + 1].mean(0), np.abs(val[0, :n - T + t + 1]).mean(0)  # [H, 2 d]
        pre, e = 0.75 * mean, 1.25 * E_MAP * size
        rms = np.sqrt((pre ** 2).mean(-1, keepdims=True) + 1e-5)
        de = np.sqrt((e ** 2).mean(-1, keepdims=True))
        bound = (e + np.abs(pre) * de / np.maximum(rms - de, 1e-9)) / rms
        over = np.abs(_np(out)[0, t] - pre / rms) - (bound + 2.0 ** -8 * (np.abs(pre / rms) + bound))
        assert over.max() <= 0, (t, over.max())


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_keep_of_a_cache_without_heads_counts(fmt):
    c = da.cache_v1(2, 20, 0, 64, fmt)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    new = i32([-7, -7])
    assert da.cache_keep(c, i32([5, 19]), i32([[0, 2], [0, 1]]), i32([2, 2]), new_lens=new) is new
    da.device_status()
    assert new.tolist() == [7, 20]


def test_a_cache_keeps_its_shapes():
    c = da.cache_v1(1, 8, 2, 64, "fp8")
    other = torch.ones((1, 8, 2), device="cuda").transpose(1, 2).contiguous()
    c.k1_scales, c.k1_scale = other, 2
    assert c.k1_scales is other and c.k1_scale == 2.0
    for name, x in (("k1", c.k1[:, :4].contiguous()), ("v", c.k1), ("k2", c.k2.cpu()), ("v_scales", other.double()),
                    ("k2", c.k2.transpose(1, 2))):
        with pytest.raises(ValueError):
            setattr(c, name, x)
    for name, x in (("n", 9), ("H", 4), ("fmt", "bf16"), ("other", 1)):
        with pytest.raises(AttributeError):
            setattr(c, name, x)
    again = copy.copy(c)
    assert again.k1 is c.k1 and again.n == 8 and copy.deepcopy(c).v.shape == c.v.shape
    with pytest.raises(AttributeError):
        da.cache_v2(1, 8, 2, 128).k2 = torch.zeros((1, 8, 2, 128), device="cuda", dtype=torch.bfloat16)


@pytest.mark.parametrize("fmt", ["bf16", "fp8k", "fp8"])
@pytest.mark.parametrize("v1,d,H", [(True, 64, 3), (False, 128, 16)])
def test_keep_moves_long_paths(v1, d, H, fmt):
    B, n, A = 4, 100, 64
    g = torch.Generator(device="cuda").manual_seed(H)
    c, _, _ = _random(g, B, n, H, d, v1, fmt)
    tensors = [t for t in (c.k1, c.k2, c.v, c.k1_scales, c.k2_scales, c.v_scales) if t is not None]
    before = [t.clone() for t in tensors]
    rs = np.random.RandomState(H)
    lens, kept = [0, 36, 20, 5], [33, 64, 50, 63]
    path = np.zeros((B, A), np.int32)
    for b in range(B):
        path[b, :kept[b]] = np.sort(rs.permutation(64)[:kept[b]])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    new = da.cache_keep(c, i32(lens), i32(path), i32(kept))
    da.device_status()
    assert new.tolist() == [x + k for x, k in zip(lens, kept)]
    for old, now in zip(before, tensors):
        want = old.clone()
        for b in range(B):
            src, dst = [lens[b] + int(x) for x in path[b, :kept[b]]], slice(lens[b], lens[b] + kept[b])
            if old.dim() == 4:
                want[b, dst] = old[b, src]
            else:
                want[b, :, dst] = old[b][:, src]
        assert torch.equal(now.view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("T", [3, 40])
def test_an_infinite_key_weighs_by_its_scores(T):
    # V1: NaN for who sees it (a map's rows meet both maps' keys); V2: nothing where its score is minus infinity
    B, H, n = 1, 2, 150
    g = torch.Generator(device="cuda").manual_seed(T)
    L, see, but = n - T, [7] * T, [5] * T
    for v1, d in ((True, 64), (False, 128)):
        c, _, _ = _random(g, B, n, H, d, v1, "bf16")
        q = [_bf(g, B, T, H if v1 else 2 * H, d) for _ in range(2)]
        for x in q:
            x[..., 0] = 1.0
        lam, logits = torch.tensor([0.25], device="cuda"), torch.randn(H, generator=g, device="cuda")

        def call(length, words):
            a = dict(lens=torch.tensor([length], dtype=torch.int32, device="cuda"),
                     mask=torch.tensor(words, dtype=torch.int64, device="cuda"))
            out = da.tree_decode(*q, c, lam, 0.2, **a) if v1 else da.v2_tree_decode(q[0], c, logits, **a)
            da.device_status()
            return out
        hidden = call(L, but)
        for x in (float("-inf"), float("inf")):
            c.k1[:, L + 1, :, 0] = x
            assert torch.equal(call(L, but), hidden)
            out = call(L, see)
            assert torch.equal(out, hidden) if x < 0 and not v1 else out.isnan().all()
        if not v1:
            c.k1[:, 1, :, 0] = float("-inf")
            assert not call(0, [2] * T).any()  # (nothing but that key)
