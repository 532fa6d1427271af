"""Rotary positions, cache append, tree decode and cache keep against fp64 references on the CPU.

Bars (derived from the formats; a rounding is off by at most finfo(t).eps / 2 relative to the value):
  * rotary: the sine and cosine are within 4 2^-24 of the exact ones (a remainder rounded to fp32, two
    ulps of sinpi / cospi, the factor), two products and a sum round once each: 8 2^-24 m (|x_a| + |x_b|),
    and the output's own rounding;
  * 8-bit rows: half an e4m3 step of the scaled value (2^-4 relative, 2^-10 absolute), plus the
    rotary error before it; scales 2^-22 relative on top of the rotary error;
  * attention: the weights stand in two terms (e4m3: 2^-4 2^-4 = 2^-8 relative, and 2^-10 absolute where
    the largest contribution is at least 2^7, 2^-17 of it a key; bf16: 2^-16, under the same bar), and 2^-10 more for
    the two-term query, exp2 and the fp32 sums: E = (2^-8 + 2^-10) sum_j p_j |v_j| (+ 2^-17 n max_j
    p_j |v_j|) on a map's output; the norm multiplies it by its gain and adds the change of the row's
    rms; the output rounds to bf16.
"""

import numpy as np
import pytest
import torch

import oracle
from differential_attention_03_gb300 import binding as da

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from differential_attention_03_gb300 import build
    build.build()
    torch.cuda.init()


def _np(t):
    return t.detach().float().cpu().double().numpy()


def _close(got, ref, bound, name):
    got = _np(got) if isinstance(got, torch.Tensor) else got
    assert np.isfinite(got).all(), f"{name}: non-finite output"
    over = np.abs(got - ref) - bound
    assert over.max(initial=-1.0) <= 0, f"{name}: {over.max()} over the bar, at {np.unravel_index(over.argmax(), over.shape)}"


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _bf(g, *shape, std=1.0):
    return (std * torch.randn(shape, generator=g, device="cuda")).to(torch.bfloat16)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ----------------------------------------------------------------------------- rotary
def _pair_sum(x, rot, inter):
    """|x_a| + |x_b| of each channel's pair (0 past rot)."""
    x = np.abs(x)
    s = np.zeros_like(x)
    if inter:
        p = x[..., 0:rot:2] + x[..., 1:rot:2]
        s[..., 0:rot:2] = s[..., 1:rot:2] = p
    else:
        p = x[..., :rot // 2] + x[..., rot // 2:rot]
        s[..., :rot // 2] = s[..., rot // 2:rot] = p
    return s


ROPE_CASES = [
    # B, n, heads, d, rot, interleaved, dtype
    (1, 1, (1,), 64, 64, False, "bf16"),
    (2, 37, (3, 3, 3, 3), 64, 64, False, "bf16"),
    (1, 300, (4, 2), 128, 64, True, "bf16"),
    (2, 9, (2, 1), 128, 128, True, "f32"),
    (1, 33, (2,), 128, 26, False, "bf16"),   # rot / 2 not a whole vector
    (1, 33, (2,), 128, 6, True, "f32"),
    (1, 65, (2, 2), 37, 30, False, "f32"),   # odd head width
    (1, 5, (1, 0, 2), 24, 16, True, "bf16"),
    (3, 700, (1,), 64, 32, False, "f32"),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("B,n,heads,d,rot,inter,dt", ROPE_CASES)
def test_rope_matches(B, n, heads, d, rot, inter, dt, inverse):
    g = _gen(n + d + rot)
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    xs = [torch.randn((B, n, h, d), generator=g, device="cuda").to(dtype) for h in heads]
    scaling, factor = [("none", 1.0), ("linear", 8.0), ("ntk", 4.0), ("yarn", 16.0)][(n + rot // 2) % 4]
    spec = da.rope_spec(rot, base=10000.0, interleaved=inter, scaling=scaling, factor=factor, original_context=4096)
    th, m = oracle.rope_frequencies(rot, 10000.0, scaling, factor, 4096)
    rs = np.random.RandomState(n)
    pos = rs.randint(-5, 2000000, (B, n)) if n % 2 else None
    got = da.rope(xs, spec, positions=None if pos is None else _i32(pos), inverse=inverse)
    da.device_status()
    pp = np.broadcast_to(np.arange(n), (B, n)) if pos is None else pos
    half = 2.0 ** -8 if dt == "bf16" else 2.0 ** -24
    for x, y in zip(xs, got):
        ref = oracle.rope(x.cpu(), pp, th, m, inter, inverse)
        f32 = 8 * 2.0 ** -24 * m * _pair_sum(_np(x), rot, inter)
        if x.numel():
            _close(y, ref, (f32 + half * (np.abs(ref) + f32)) * (1 + 1e-9), "rope")
            assert torch.equal(y[..., rot:], x[..., rot:])
    # in place: the same bits
    again = [x.clone() for x in xs]
    out = da.rope(again, spec, positions=None if pos is None else _i32(pos), inverse=inverse, out=again)
    assert all(torch.equal(a, b) for a, b in zip(out, got))


def test_rope_far_positions_are_exact():
    # The phase wraps in integers: at the ends of int32 the error is still that of fp32 sines.
    th, m = oracle.rope_frequencies(64)
    spec = da.rope_spec(64)
    pos = np.array([[0, 1, 2 ** 20 + 1, 2 ** 31 - 1, -2 ** 31, -1]])
    x = torch.ones((1, 6, 1, 64), device="cuda")
    y = da.rope([x], spec, positions=_i32(pos))[0]
    # (the frequencies are doubles: 2^31 positions of one off by 2^-53 is 2^-22)
    _close(y, oracle.rope(x.cpu(), pos, th, m), 16 * 2.0 ** -24 + 2.0 ** -21, "far rope")


def test_rope_backward_is_the_gradient():
    # <dy, R(x + h e) - R(x - h e)> / 2h against the inverse rotation of dy, in fp64 on the oracle and by the kernel
    rot, d, n = 16, 24, 5
    th, m = oracle.rope_frequencies(rot, scaling="yarn", factor=4.0, original=64)
    spec = da.rope_spec(rot, scaling="yarn", factor=4.0, original_context=64)
    g = _gen(3)
    x, dy = (torch.randn((1, n, 2, d), generator=g, device="cuda") for _ in range(2))
    dx = da.rope([dy], spec, inverse=True)[0]
    pos = np.arange(n)[None]
    xn, dyn = _np(x), _np(dy)
    num = np.zeros_like(xn)
    for i in np.ndindex(*xn.shape):
        e = np.zeros_like(xn)
        e[i] = 0.5
        num[i] = (dyn * (oracle.rope(xn + e, pos, th, m) - oracle.rope(xn - e, pos, th, m))).sum()
    _close(dx, num, 9 * 2.0 ** -24 * m * _pair_sum(dyn, rot, False) + 2.0 ** -23 * np.abs(num) + 1e-12, "gradient")


# ----------------------------------------------------------------------------- caches
def _random_cache(g, B, n, H, d, v1, fmt, spread=0.5):
    """A cache with contents, and its values in fp64: (cache, keys, values)."""
    dv = 2 * d if v1 else d
    ks = (0.013, 0.021)
    c = da.cache_v1(B, n, H, d, fmt, k1_scale=ks[0], k2_scale=ks[1]) if v1 else da.cache_v2(B, n, H, d, fmt, k_scale=ks[0])
    keys = []
    for i, t in enumerate([c.k1] + ([c.k2] if v1 else [])):
        x = torch.randn((B, n, H, d), generator=g, device="cuda")
        if fmt == "bf16":
            t.copy_(x)
            keys.append(_np(t))
        elif fmt == "fp8k":
            t.copy_((x / ks[i]).clamp(-448, 448))
            keys.append(_np(t) * ks[i])
        else:
            keys.append(_fill_rows(t, (c.k1_scales, c.k2_scales)[i], x))
    x = torch.randn((B, n, H, dv), generator=g, device="cuda")
    x = x * torch.exp(spread * torch.randn((B, n, H, 1), generator=g, device="cuda"))
    if fmt == "fp8":
        val = _fill_rows(c.v, c.v_scales, x)
    else:
        c.v.copy_(x)
        val = _np(c.v)
    return c, keys, val


def _fill_rows(codes, scales, x):
    s = x.abs().amax(-1) / 448.0
    codes.copy_((x / s.unsqueeze(-1)).clamp(-448, 448))
    scales.copy_(s.transpose(1, 2))
    return _np(codes) * _np(s)[..., None]


def _contents(c):
    return [t.clone() for t in (c.k1, c.k2, c.v, c.k1_scales, c.k2_scales, c.v_scales) if t is not None]


def _same(a, b):
    return all(torch.equal(x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x,
                           y.view(torch.uint8) if y.dtype == torch.float8_e4m3fn else y) for x, y in zip(a, b))


# v1, B, T, H, Hq, d, n, rot, interleaved, lens, ntok
APPEND_CASES = [
    (True, 1, 1, 1, 1, 64, 3, 64, False, [2], None),
    (True, 3, 1, 5, 5, 128, 40, 128, True, [0, 39, 17], None),
    (True, 2, 70, 3, 3, 64, 200, 32, False, [130, 0], [70, 13]),
    (True, 2, 33, 2, 2, 128, 64, 22, False, [31, 60], [33, 33]),      # the second runs past the cache
    (False, 2, 19, 2, 4, 128, 50, 64, True, [0, 31], [0, 19]),
    (False, 1, 300, 1, 8, 128, 300, 128, False, None, None),
    (False, 2, 5, 3, 6, 128, 16, 0, False, [-3, 14], [5, 7]),         # rows before the cache, no rotation
]


@pytest.mark.parametrize("fmt", ["bf16", "fp8k", "fp8"])
@pytest.mark.parametrize("v1,B,T,H,Hq,d,n,rot,inter,lens,ntok", APPEND_CASES)
def test_append_matches(v1, B, T, H, Hq, d, n, rot, inter, lens, ntok, fmt):
    g = _gen(T + n + rot)
    c, _, _ = _random_cache(g, B, n, H, d, v1, fmt)
    before = _contents(c)
    q = [_bf(g, B, T, Hq, d) for _ in range(2 if v1 else 1)]
    k = [_bf(g, B, T, H, d, std=2.0) for _ in range(2 if v1 else 1)]
    v = _bf(g, B, T, H, 2 * d if v1 else d)
    k[0][0, 0, 0] = 0  # a row of zeros
    rs = np.random.RandomState(T)
    pos = rs.randint(0, 100000, (B, T)) if T % 2 else None
    spec = da.rope_spec(rot, interleaved=inter) if rot else None
    a = dict(rope=spec, positions=None if pos is None else _i32(pos), lens=None if lens is None else _i32(lens),
             ntok=None if ntok is None else _i32(ntok))
    if v1:
        qo = da.cache_append(c, *k, v, q1=q[0], q2=q[1], **a)
    else:
        qo = [da.v2_cache_append(c, *k, v, q=q[0], **a)]
    da.device_status()
    th, m = oracle.rope_frequencies(rot) if rot else (np.zeros(0), 1.0)
    L = np.zeros(B, int) if lens is None else np.array(lens)
    nt = np.full(B, T) if ntok is None else np.minimum(ntok, T)
    rows = L[:, None] + np.arange(T)
    pp = rows if pos is None else pos
    for x, y in zip(q, qo):
        ref = oracle.rope(x.cpu(), pp, th, m, inter)
        f32 = 8 * 2.0 ** -24 * m * _pair_sum(_np(x), rot, inter)
        for b in range(B):
            ref[b, nt[b]:] = f32[b, nt[b]:] = 0
        _close(y, ref, (f32 + 2.0 ** -8 * (np.abs(ref) + f32)) * (1 + 1e-9), "queries")
    tensors = [(c.k1, c.k1_scales, c.k1_scale, k[0], True)]
    if v1:
        tensors.append((c.k2, c.k2_scales, c.k2_scale, k[1], True))
    tensors.append((c.v, c.v_scales, 1.0, v, False))
    written = np.zeros((B, n), bool)
    for t, scales, scale, x, key in tensors:
        ref = oracle.rope(x.cpu(), pp, th, m, inter) if key else _np(x)
        err = 8 * 2.0 ** -24 * m * _pair_sum(_np(x), rot, inter) if key else np.zeros_like(ref)
        got = _np(t)
        for b in range(B):
            for tt in range(nt[b]):
                r = L[b] + tt
                if not 0 <= r < n:
                    continue
                written[b, r] = True
                y, e = ref[b, tt], err[b, tt]
                if t.dtype == torch.bfloat16:
                    _close(got[b, r], y, (e + 2.0 ** -8 * (np.abs(y) + e)) * (1 + 1e-9), "row")
                    continue
                if fmt == "fp8k":
                    s = np.full((y.shape[0], 1), scale)
                    es = np.zeros_like(s)
                else:
                    s = _np(scales)[b, :, r][:, None]
                    sr = np.abs(y).max(-1, keepdims=True) / 448
                    es = e.max(-1, keepdims=True) / 448 + 2.0 ** -22 * sr
                    _close(s, sr, es, "scale")
                sat = np.clip(y, -448 * s, 448 * s)
                _close(got[b, r] * s, sat, (e + 448 * es) + 2.0 ** -4 * np.abs(sat) * (1 + 1e-6) + 2.0 ** -10 * s * 1.001, "codes")
    # every other row keeps its bits
    keep = torch.tensor(~written, device="cuda")
    for old, new in zip(before, _contents(c)):
        if old.dtype == torch.float8_e4m3fn:
            old, new = old.view(torch.uint8), new.view(torch.uint8)
        kk = keep[:, :, None, None] if old.dim() == 4 else keep[:, None, :]
        assert torch.equal(torch.where(kk, old, 0), torch.where(kk, new, 0))


def test_append_rows_with_non_finite_values_read_as_nan():
    c = da.cache_v1(1, 4, 2, 64, "fp8")
    g = _gen(5)
    k1, k2, v = _bf(g, 1, 3, 2, 64), _bf(g, 1, 3, 2, 64), _bf(g, 1, 3, 2, 128)
    v[0, 0, 0, 7], v[0, 1, 1, 100], k1[0, 2, 0, 3] = float("nan"), float("inf"), float("-inf")
    da.cache_append(c, k1, k2, v)
    da.device_status()
    vals = c.v.float() * c.v_scales.transpose(1, 2).unsqueeze(-1)
    keys = c.k1.float() * c.k1_scales.transpose(1, 2).unsqueeze(-1)
    nan_v, nan_k = vals.isnan().all(-1), keys.isnan().all(-1)
    assert nan_v[0, 0].tolist() == [True, False] and nan_v[0, 1].tolist() == [False, True]
    assert nan_k[0, 2].tolist() == [True, False]
    assert not vals[0, 2].isnan().any() and not keys[0, :2].isnan().any()


def test_append_tiny_and_huge_rows():
    # magnitudes at both ends of bf16: the scale stays a normal number, values stay within half a step
    c = da.cache_v2(1, 4, 1, 128, "fp8")
    g = _gen(6)
    base = torch.randn((1, 4, 1, 128), generator=g, device="cuda")
    x = (base * torch.tensor([1e-38, 1e-30, 1e30, 1e37], device="cuda").view(1, 4, 1, 1)).to(torch.bfloat16)
    da.v2_cache_append(c, x, x)
    da.device_status()
    s = _np(c.v_scales)[0, 0]
    _close(_np(c.v)[0, :, 0] * s[:, None], _np(x)[0, :, 0], 2.0 ** -4 * np.abs(_np(x)[0, :, 0]) * 1.0001 + 2.0 ** -10 * s[:, None] * 1.001,
           "rows")


# ----------------------------------------------------------------------------- tree decode
def _tree_mask(rs, T):
    """Ancestor words of a random tree."""
    words = []
    for j in range(T):
        w = 1 << j
        if j and rs.rand() < 0.85:
            w |= words[rs.randint(max(0, j - 4), j)]
        words.append(w)
    return words


def _words(mask):
    return torch.tensor(np.array(mask, dtype=np.uint64).astype(np.int64), device="cuda")


def _case_v1(B, T, H, d, n, lens, ntok, masked, fmt, seed, spread=0.5, workspace=None):
    g, rs = _gen(seed), np.random.RandomState(seed)
    c, keys, val = _random_cache(g, B, n, H, d, True, fmt, spread)
    q1, q2 = _bf(g, B, T, H, d), _bf(g, B, T, H, d)
    gamma = 0.9 + 0.2 * torch.rand(2 * d, generator=g, device="cuda")
    lam = torch.tensor([0.37], device="cuda")
    mask = [_tree_mask(rs, T) for _ in range(B)] if masked else None
    out = da.tree_decode(q1, q2, c, lam, 0.3, gamma=gamma, lens=None if lens is None else _i32(lens),
                         ntok=None if ntok is None else _i32(ntok), mask=None if mask is None else _words(mask),
                         workspace=workspace)
    da.device_status()
    L = [max(0, min(n, x)) for x in (lens or [n - T] * B)]
    nt = [max(0, min(T, x)) for x in (ntok or [T] * B)]
    ref, pre, spr, top, gain = oracle.tree_v1(q1.cpu(), q2.cpu(), *keys, val, L, nt, mask, float(lam.item()), 0.3,
                                              gamma.cpu(), 1e-5)
    e = (2.0 ** -8 + 2.0 ** -10) * spr
    if fmt == "fp8":
        e = e + 2.0 ** -17 * n * top[..., None]
    rms = np.sqrt((pre ** 2).mean(-1, keepdims=True) + 1e-5)
    de = np.sqrt((e ** 2).mean(-1, keepdims=True))
    bound = gain * (e + np.abs(pre) * de / np.maximum(rms - de, 1e-9)) * 1.1
    _close(out, ref, bound + 2.0 ** -8 * (np.abs(ref) + bound) + 1e-30, "tree v1")
    return out, ref


V1_CASES = [
    # B, T, H, d, n, lens, ntok, masked
    (1, 1, 1, 64, 1, None, None, False),
    (1, 1, 2, 128, 128, None, None, False),
    (2, 1, 3, 64, 700, [699, 5], None, False),
    (2, 5, 3, 64, 300, [295, 0], [5, 3], True),
    (1, 33, 2, 128, 400, [300], None, True),
    (2, 64, 2, 64, 200, [136, 64], [64, 50], True),
    (3, 7, 2, 128, 260, [253, 256, -4], [7, 7, 7], True),   # the second's drafts run past the cache
    (2, 64, 1, 128, 129, [65, 10], [64, 0], False),          # a sequence without drafts
    (4, 2, 1, 64, 256, [0, 127, 128, 129], [2, 1, 2, 0], True),
]


@pytest.mark.parametrize("fmt", ["bf16", "fp8k", "fp8"])
@pytest.mark.parametrize("B,T,H,d,n,lens,ntok,masked", V1_CASES)
def test_tree_v1_matches(B, T, H, d, n, lens, ntok, masked, fmt):
    _case_v1(B, T, H, d, n, lens, ntok, masked, fmt, seed=n + T)


V2_CASES = [
    # B, T, Hq, Hkv, n, lens, ntok, masked, logits' dimensions
    (1, 1, 2, 1, 1, None, None, False, 1),
    (2, 1, 8, 2, 500, [499, 0], None, False, 2),
    (2, 5, 8, 2, 300, [295, 11], [5, 4], True, 3),
    (1, 64, 4, 1, 333, [200], None, True, 3),    # two row tiles a key head
    (2, 20, 16, 2, 150, [130, 77], [20, 1], True, 3),  # three pairs a tile, four pairs a head
    (1, 33, 2, 1, 1000, [900], None, False, 1),
]


@pytest.mark.parametrize("fmt", ["bf16", "fp8k", "fp8"])
@pytest.mark.parametrize("B,T,Hq,Hkv,n,lens,ntok,masked,ldim", V2_CASES)
def test_tree_v2_matches(B, T, Hq, Hkv, n, lens, ntok, masked, ldim, fmt):
    d = 128
    g, rs = _gen(n + T), np.random.RandomState(n + T)
    c, keys, val = _random_cache(g, B, n, Hkv, d, False, fmt)
    q = _bf(g, B, T, Hq, d)
    logits = torch.randn((B, T, Hq // 2)[3 - ldim:] if ldim != 2 else (B, Hq // 2), generator=g, device="cuda")
    mask = [_tree_mask(rs, T) for _ in range(B)] if masked else None
    scale = 0.11 if T == 20 else 0.0
    out = da.v2_tree_decode(q, c, logits, lens=None if lens is None else _i32(lens),
                            ntok=None if ntok is None else _i32(ntok), mask=None if mask is None else _words(mask),
                            softmax_scale=scale)
    da.device_status()
    L = [max(0, min(n, x)) for x in (lens or [n - T] * B)]
    nt = [max(0, min(T, x)) for x in (ntok or [T] * B)]
    lg = _np(logits)
    lg = np.broadcast_to(lg[:, None] if ldim == 2 else lg, (B, T, Hq // 2))
    ref, spr, top = oracle.tree_v2(q.cpu(), keys[0], val, lg, L, nt, mask, scale or None)
    e = (2.0 ** -8 + 2.0 ** -10) * spr
    if fmt == "fp8":
        e = e + 2.0 ** -17 * n * top[..., None]
    _close(out, ref, e + 2.0 ** -8 * (np.abs(ref) + e) + 1e-30, "tree v2")


def test_tree_token_that_sees_nothing_is_zero():
    out, _ = _case_v1(2, 4, 2, 64, 130, [0, 126], [4, 0], False, "bf16", 11)
    assert torch.count_nonzero(out[1]) == 0  # (no drafts)
    g = _gen(12)
    for fmt in ("bf16", "fp8"):
        c, _, _ = _random_cache(g, 1, 130, 2, 64, True, fmt)
        q = _bf(g, 1, 3, 2, 64)
        lam = torch.tensor([0.4], device="cuda")
        out = da.tree_decode(q, q, c, lam, 0.2, lens=_i32([0]), mask=_words([0, 2, 0]))
        da.device_status()
        assert torch.count_nonzero(out[0, 0]) == 0 and torch.count_nonzero(out[0, 2]) == 0
        assert torch.isfinite(out).all() and torch.count_nonzero(out[0, 1]) > 0
        empty = da.cache_v1(1, 0, 2, 64, fmt)
        out = da.tree_decode(q, q, empty, lam, 0.2, lens=_i32([0]))
        da.device_status()
        assert torch.count_nonzero(out) == 0


@pytest.mark.parametrize("fmt", ["bf16", "fp8k", "fp8"])
@pytest.mark.parametrize("v1,T,R", [(True, 5, 64), (True, 40, 128), (False, 9, 128)])
def test_tree_is_blind_to_what_it_must_not_see(v1, T, R, fmt):
    # Rows behind the drafts, a hidden draft and rows of other sequences hold NaN and infinities.
    d, n, H, B = R, 300, 2, 2
    g = _gen(T)
    c, _, _ = _random_cache(g, B, n, H, d, v1, fmt)
    lens, ntok = [200, 250], [T, T - 2]
    mask = np.tril(np.ones((T, T), int))
    mask[:, 1] = 0  # draft 1 is seen by itself alone
    mask[1, 1] = 1
    words = [sum(int(b) << u for u, b in enumerate(r)) for r in mask]
    q = [_bf(g, B, T, H if v1 else 4 * H, d) for _ in range(2)]
    lam = torch.tensor([0.4], device="cuda")
    logits = torch.randn(2 * H, generator=g, device="cuda")

    def call():
        a = dict(lens=_i32(lens), ntok=_i32(ntok), mask=_words(words))
        out = da.tree_decode(*q, c, lam, 0.2, **a) if v1 else da.v2_tree_decode(q[0], c, logits, **a)
        da.device_status()
        return out
    clean = call()
    assert torch.isfinite(clean).all()
    bad = {torch.bfloat16: [float("nan"), float("inf"), float("-inf")], torch.float8_e4m3fn: [float("nan")] * 3}
    for t in [c.k1, c.v] + ([c.k2] if v1 else []):
        for b in range(B):
            end = lens[b] + ntok[b]
            for i, x in enumerate(bad[t.dtype]):
                t[b, end + i::3] = x
            t[b, lens[b] + 1, :, 3:9] = bad[t.dtype][b]
    if fmt == "fp8":
        for s in [c.k1_scales, c.v_scales] + ([c.k2_scales] if v1 else []):
            for b in range(B):
                s[b, :, lens[b] + ntok[b]:] = float("nan")
                s[b, :, lens[b] + 1] = float("inf")
    out = call()
    others = [t for t in range(T) if t != 1]
    assert torch.equal(out[:, others], clean[:, others])
    assert out[:, 1].isnan().all()  # and whoever sees it, sees it


@pytest.mark.parametrize("fmt", ["bf16", "fp8k", "fp8"])
@pytest.mark.parametrize("B,T,H,d,n,lens", [(1, 3, 1, 64, 40000, [39997]), (1, 2, 3, 128, 20000, [19990]),
                                            (37, 4, 5, 64, 400, None), (150, 1, 1, 128, 130, None)])
def test_tree_many_tiles_and_many_units(B, T, H, d, n, lens, fmt):
    rs = np.random.RandomState(n)
    if lens is None:
        lens = [int(x) for x in rs.randint(0, n - T, B)]
    _case_v1(B, T, H, d, n, lens, None, True, fmt, seed=n + B)


@pytest.mark.parametrize("fmt", ["bf16", "fp8k", "fp8"])
@pytest.mark.parametrize("v1,T,H,d", [(True, 1, 12, 128), (True, 16, 12, 128), (True, 40, 6, 128), (True, 1, 8, 64),
                                      (True, 24, 6, 64), (False, 1, 8, 128), (False, 12, 8, 128)])
def test_tree_gives_the_same_bits_again(v1, T, H, d, fmt):
    # Long ragged caches whose last tiles end at every place: a value tile is cleaned while earlier ones
    # are still in the ring, and nothing of that may show.
    n, lens = 6000, [5187, 4096 - T, 3007, 4762]
    g = _gen(T + d)
    c, _, _ = _random_cache(g, 4, n, H, d, v1, fmt)
    q = [_bf(g, 4, T, H if v1 else 2 * H, d) for _ in range(2)]
    lam, logits = torch.tensor([0.4], device="cuda"), torch.randn(H, generator=g, device="cuda")

    def call(b=None):
        cut = c if b is None else da.KVCache(fmt, *(None if t is None else t[b:b + 1] for t in (c.k1, c.k2, c.v)), c.k1_scale,
                                             c.k2_scale, *(None if t is None else t[b:b + 1] for t in (c.k1_scales, c.k2_scales, c.v_scales)))
        qq = q if b is None else [x[b:b + 1] for x in q]
        ll = _i32(lens if b is None else lens[b:b + 1])
        return da.tree_decode(*qq, cut, lam, 0.2, lens=ll) if v1 else da.v2_tree_decode(qq[0], cut, logits, lens=ll)
    first = call()
    assert all(torch.equal(first, call()) for _ in range(12))
    da.device_status()
    # and a sequence alone, its keys dealt out otherwise, is the same up to the bars of both
    for b in range(4):
        err = (call(b)[0].float() - first[b].float()).abs().max()
        assert err <= 2e-2 * max(1.0, float(first[b].abs().max()))
    da.device_status()


@pytest.mark.parametrize("fmt", ["bf16", "fp8k", "fp8"])
def test_tree_climbing_scores_and_a_sink(fmt):
    # Scores that climb along the cache (the reference maximum moves all the way), and one key that
    # takes most of the weight with a value row 2^-20 of the others'.
    B, T, H, d, n = 1, 4, 2, 64, 3000
    g = _gen(77)
    c, keys, val = _random_cache(g, B, n, H, d, True, fmt)
    q1, q2 = _bf(g, B, T, H, d), _bf(g, B, T, H, d)
    q1[:] = q1[:, :1]
    dirs = q1[0, 0].float() / q1[0, 0].float().norm(dim=-1, keepdim=True)
    k1 = dirs * torch.linspace(0, 25, n, device="cuda").view(1, n, 1, 1) + 0.3 * torch.randn((1, n, H, d), generator=g, device="cuda")
    k2 = torch.randn((1, n, H, d), generator=g, device="cuda")
    k2[:, 100] = 8 * q2[:, 0].float() / q2[:, 0].float().norm(dim=-1, keepdim=True)
    v = torch.randn((1, n, H, 2 * d), generator=g, device="cuda")
    v[:, 100] *= 2.0 ** -20
    if fmt == "fp8":
        keys = [_fill_rows(c.k1, c.k1_scales, k1), _fill_rows(c.k2, c.k2_scales, k2)]
        val = _fill_rows(c.v, c.v_scales, v)
    else:
        for i, (t, k, s) in enumerate(((c.k1, k1, 0.06), (c.k2, k2, 0.03))):
            if fmt == "bf16":
                t.copy_(k)
                keys[i] = _np(t)
            else:
                t.copy_((k / s).clamp(-448, 448))
                keys[i] = _np(t) * s
        c.k1_scale, c.k2_scale = 0.06, 0.03
        c.v.copy_(v)
        val = _np(c.v)
    out = da.tree_decode(q1, q2, c, torch.tensor([0.37], device="cuda"), 0.3)
    da.device_status()
    ref, pre, spr, top, gain = oracle.tree_v1(q1.cpu(), q2.cpu(), *keys, val, [n - T], [T], None,
                                              float(np.float32(0.37)), 0.3, np.ones(2 * d), 1e-5)
    e = (2.0 ** -8 + 2.0 ** -10) * spr + (2.0 ** -17 * n * top[..., None] if fmt == "fp8" else 0)
    # (scores of up to 30 powers of e: fp32's sums of products are off by 2^-24 of 64 such terms)
    e = e + 30 * 64 * 2.0 ** -24 * spr
    rms = np.sqrt((pre ** 2).mean(-1, keepdims=True) + 1e-5)
    de = np.sqrt((e ** 2).mean(-1, keepdims=True))
    bound = gain * (e + np.abs(pre) * de / np.maximum(rms - de, 1e-9)) * 1.1
    _close(out, ref, bound + 2.0 ** -8 * (np.abs(ref) + bound), "tree")


def test_tree_of_one_token_is_the_decode_step():
    # the existing one-token calls over the same bf16 and fp8k caches: both within their bars of the
    # same number, so within two roundings of bf16 and twice the weights' of each other
    B, H, d, n = 3, 4, 64, 900
    g = _gen(8)
    lens = [900, 5, 333]
    for fmt in ("bf16", "fp8k"):
        c, _, _ = _random_cache(g, B, n, H, d, True, fmt)
        q1, q2 = _bf(g, B, 1, H, d), _bf(g, B, 1, H, d)
        lam = torch.tensor([0.3], device="cuda")
        a = da.tree_decode(q1, q2, c, lam, 0.4, lens=_i32([x - 1 for x in lens]))
        if fmt == "bf16":
            b = da.diffattn_decode(q1[:, 0].contiguous(), q2[:, 0].contiguous(), c.k1, c.k2, c.v, lam, 0.4, lens=_i32(lens))
        else:
            b = da.diffattn_decode_fp8k(q1[:, 0].contiguous(), q2[:, 0].contiguous(), c.k1, c.k2, c.k1_scale, c.k2_scale,
                                        c.v, lam, 0.4, lens=_i32(lens))
        da.device_status()
        a, b = _np(a)[:, 0], _np(b)
        assert np.abs(a - b).max() <= 2e-2 * max(1.0, np.abs(b).max())


# ----------------------------------------------------------------------------- keep
@pytest.mark.parametrize("fmt", ["bf16", "fp8k", "fp8"])
@pytest.mark.parametrize("v1,d,H,n", [(True, 64, 3, 40), (True, 128, 16, 90), (False, 128, 1, 70)])
def test_keep_moves_the_path(v1, d, H, n, fmt):
    B, A = 6, 12
    g = _gen(n)
    c, _, _ = _random_cache(g, B, n, H, d, v1, fmt)
    before = _contents(c)
    lens = [0, 3, n - 8, n, 10, -2]
    path = [[0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11],   # in place
            [0, 2, 3, 5, 8, 9, 10, 11, 12, 13, 14, 15],
            [1, 2, 4, 7, 9, 10, 11, 12, 13, 14, 15, 16],  # runs past the cache: cut after 7
            [0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11],   # no room at all
            [2, 3, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12],   # does not ascend: two nodes
            [0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11]]   # before the cache
    nkeep = [12, 9, 12, 5, 12, 3]
    kept = [12, 9, 4, 0, 2, 0]
    new = da.cache_keep(c, _i32(lens), _i32(path), _i32(nkeep))
    da.device_status()
    assert new.tolist() == [x + k for x, k in zip(lens, kept)]
    for old, now in zip(before, _contents(c)):
        if old.dtype == torch.float8_e4m3fn:
            old, now = old.view(torch.uint8), now.view(torch.uint8)
        want = old.clone()
        for b in range(B):
            for i in range(kept[b]):
                if old.dim() == 4:
                    want[b, lens[b] + i] = old[b, lens[b] + path[b][i]]
                else:
                    want[b, :, lens[b] + i] = old[b, :, lens[b] + path[b][i]]
        assert torch.equal(now, want)


# ----------------------------------------------------------------------------- together
def _step(c, x, st, spec, T):
    """One speculative step: append the drafts, attend, keep the path."""
    q1, q2 = da.cache_append(c, x["k1"], x["k2"], x["v"], q1=x["q1"], q2=x["q2"], rope=spec,
                             positions=st["pos"], lens=st["lens"], ntok=st["ntok"])
    out = da.tree_decode(q1, q2, c, st["lam"], 0.3, lens=st["lens"], ntok=st["ntok"], mask=st["mask"])
    new = da.cache_keep(c, st["lens"], st["path"], st["nkeep"])
    return out, new


def _speculative(g, B, T, H, d):
    return {"q1": _bf(g, B, T, H, d), "q2": _bf(g, B, T, H, d), "k1": _bf(g, B, T, H, d), "k2": _bf(g, B, T, H, d),
            "v": _bf(g, B, T, H, 2 * d)}


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_speculative_decoding_equals_plain_decoding(fmt):
    # A prefill, then drafted trees of which one path is accepted each time, then a plain step; the
    # plain step's output is compared with the fp64 attention of the accepted tokens alone, rotated at
    # their positions.
    B, H, d, T, n0 = 2, 3, 64, 6, 50
    g = _gen(99)
    spec = da.rope_spec(d, scaling="linear", factor=2.0)
    th, m = oracle.rope_frequencies(d, scaling="linear", factor=2.0)
    c = da.cache_v1(B, 120, H, d, fmt)
    pre = _speculative(g, B, n0, H, d)
    da.cache_append(c, pre["k1"], pre["k2"], pre["v"], rope=spec, ntok=_i32([50, 31]))
    lens = [50, 31]
    seqs = [{k: [pre[k][b, t] for t in range(lens[b])] for k in ("k1", "k2", "v")} for b in range(B)]
    lam = torch.tensor([0.4], device="cuda")
    parent = [-1, 0, 0, 1, 2, 4]
    depth = [0, 1, 1, 2, 2, 3]
    words = []
    for j, p in enumerate(parent):
        words.append((1 << j) | (words[p] if p >= 0 else 0))
    for path in ([[0, 2, 4, 5], [0, 1, 3]], [[0], [0, 2, 4]]):
        x = _speculative(g, B, T, H, d)
        st = {"pos": _i32([[L + e for e in depth] for L in lens]), "lens": _i32(lens), "ntok": _i32([6, 5]),
              "mask": _words(words), "lam": lam, "path": _i32([p + [0] * (T - len(p)) for p in path]),
              "nkeep": _i32([len(p) for p in path])}
        _, new = _step(c, x, st, spec, T)
        da.device_status()
        for b in range(B):
            for k in seqs[b]:
                seqs[b][k] += [x[k][b, u] for u in path[b]]
            lens[b] += len(path[b])
        assert new.tolist() == lens
    x = _speculative(g, B, 1, H, d)
    q1, q2 = da.cache_append(c, x["k1"], x["k2"], x["v"], q1=x["q1"], q2=x["q2"], rope=spec, lens=_i32(lens))
    out = da.tree_decode(q1, q2, c, lam, 0.3, lens=_i32(lens))
    da.device_status()
    for b in range(B):
        full = {k: torch.stack(seqs[b][k] + [x[k][b, 0]])[None] for k in seqs[b]}
        n = lens[b] + 1
        pos = np.arange(n)[None]
        vals = {}
        for k in ("k1", "k2"):
            y = oracle.rope(full[k].cpu(), pos, th, m)
            if fmt == "bf16":
                vals[k] = _np(torch.tensor(y).to(torch.bfloat16))
            else:
                codes, s = oracle.quantise_rows(y)
                vals[k] = codes * s[..., None]
        vals["v"] = _np(full["v"])
        if fmt == "fp8":
            codes, s = oracle.quantise_rows(vals["v"])
            vals["v"] = codes * s[..., None]
        qq = [oracle.rope(x[k][b:b + 1].cpu(), np.array([[lens[b]]]), th, m) for k in ("q1", "q2")]
        ref = oracle.diff_attn_v1_decode(qq[0][:, 0], qq[1][:, 0], vals["k1"], vals["k2"], vals["v"], 0.4, 0.3,
                                         np.ones(2 * d), 1e-5)
        # (the rotated query is rounded to bf16, 2^-8 of its scores; codes near a tie may fall either way)
        assert np.abs(_np(out)[b, 0] - ref[0]).max() <= 3e-2 * max(1.0, np.abs(ref).max())


def test_chain_of_drafts_equals_the_causal_forward():
    # A 60-token prompt and 40 drafted tokens in a chain against diffattn_forward over the 100 rotated tokens.
    B, H, d, n, T = 2, 2, 64, 100, 40
    g = _gen(15)
    x = _speculative(g, B, n, H, d)
    spec = da.rope_spec(d, interleaved=True)
    q1, q2, k1, k2 = da.rope([x["q1"], x["q2"], x["k1"], x["k2"]], spec)
    lam = torch.tensor([0.4], device="cuda")
    ref = da.diffattn_forward(q1, q2, k1, k2, x["v"], lam, 0.3)
    c = da.cache_v1(B, n, H, d)
    cut = lambda t, a, b: t[:, a:b].contiguous()  # noqa: E731
    da.cache_append(c, cut(x["k1"], 0, 60), cut(x["k2"], 0, 60), cut(x["v"], 0, 60), rope=spec)
    qa, qb = da.cache_append(c, cut(x["k1"], 60, n), cut(x["k2"], 60, n), cut(x["v"], 60, n), q1=cut(x["q1"], 60, n),
                             q2=cut(x["q2"], 60, n), rope=spec, lens=_i32([60, 60]))
    out = da.tree_decode(qa, qb, c, lam, 0.3, lens=_i32([60, 60]))
    da.device_status()
    assert torch.equal(c.k1, k1) and torch.equal(c.k2, k2) and torch.equal(c.v, x["v"])
    assert torch.equal(qa, cut(q1, 60, n)) and torch.equal(qb, cut(q2, 60, n))
    a, b = _np(out), _np(ref)[:, 60:]
    assert np.abs(a - b).max() <= 2e-2 * max(1.0, np.abs(b).max())


def test_bf16_weights_lose_nothing():
    # 8000 alike keys: the output is off by its own rounding (uniform, at most 2^-8 of the value's power of
    # two: 2^-8 / sqrt 3, over 1.44 rms: 1.6e-3 of the norm); weights in one bf16 term alone would make it 2.4e-3.
    B, T, H, d, n = 1, 4, 2, 64, 8000
    g = _gen(5)
    c, keys, val = _random_cache(g, B, n, H, d, True, "bf16")
    q1, q2 = _bf(g, B, T, H, d), _bf(g, B, T, H, d)
    out = da.tree_decode(q1, q2, c, torch.tensor([0.4], device="cuda"), 0.3)
    da.device_status()
    ref = oracle.tree_v1(q1.cpu(), q2.cpu(), *keys, val, [n - T], [T], None, float(np.float32(0.4)), 0.3, np.ones(2 * d),
                         1e-5)[0]
    assert np.linalg.norm(_np(out) - ref) <= 2.0e-3 * np.linalg.norm(ref)


def test_offsets_past_32_bits():
    # Caches of 2^32 and more values, e4m3: rows near their end are written, found, and moved.
    n, H, d, T = 2 ** 21 + 5000, 16, 128, 4
    g = _gen(21)
    c = da.cache_v2(1, n, H, d, "fp8")
    L = n - 40
    k, v = _bf(g, 1, T, H, d), _bf(g, 1, T, H, d)
    da.v2_cache_append(c, k, v, lens=_i32([L - T]))          # committed rows, far in
    da.v2_cache_append(c, _bf(g, 1, 8, H, d), v.repeat(1, 2, 1, 1), lens=_i32([L]))
    da.device_status()
    for t, s, x in ((c.k1, c.k1_scales, k), (c.v, c.v_scales, v)):
        codes, scale = oracle.quantise_rows(x.cpu())
        back = _np(t[:, L - T:L]) * _np(s[:, :, L - T:L]).transpose(0, 2, 1)[..., None]
        assert np.abs(back - _np(x)).max() <= (2.0 ** -4 + 2.0 ** -10) * np.abs(_np(x)).max()
    assert not c.k1[0, :L - T].view(torch.uint8).any() and not c.v[0, L + 8:].view(torch.uint8).any()
    # a query along one far key (every other key but the drafts' is zero): its value is the output
    q = (4 * k[:, 1:2].float().repeat_interleave(2, 2)).to(torch.bfloat16)
    logits = torch.zeros(H, device="cuda")
    out = da.v2_tree_decode(q, c, logits, lens=_i32([L]), ntok=_i32([1]), mask=torch.zeros(1, dtype=torch.int64, device="cuda"))
    da.device_status()
    ref = 0.5 * _np(c.v[:, L - T + 1:L - T + 2]) * _np(c.v_scales[:, :, L - T + 1:L - T + 2]).transpose(0, 2, 1)[..., None]
    # (q.k / sqrt d is 4 |k|^2 / 11.3, some 45 of e: what 2^21 zero keys and three others weigh is below 2^-30)
    assert np.abs(_np(out) - ref).max() <= 2.0 ** -6 * np.abs(ref).max()
    rows = c.k1[0, [L + 1, L + 3, L + 7]].view(torch.uint8).clone(), c.v_scales[0, :, [L + 1, L + 3, L + 7]].clone()
    new = da.cache_keep(c, _i32([L]), _i32([[1, 3, 7]]), _i32([3]))
    da.device_status()
    assert new.tolist() == [L + 3]
    assert torch.equal(c.k1[0, L:L + 3].view(torch.uint8), rows[0]) and torch.equal(c.v_scales[0, :, L:L + 3], rows[1])


def test_rope_past_32_bits():
    n, H, d = 2 ** 21 + 777, 16, 128
    x = torch.zeros((1, n, H, d), device="cuda", dtype=torch.bfloat16)
    x[:, -3:] = _bf(_gen(4), 1, 3, H, d)
    last = x[:, -3:].clone()
    th, m = oracle.rope_frequencies(d)
    da.rope([x], da.rope_spec(d), out=[x])
    da.device_status()
    ref = oracle.rope(last.cpu(), np.arange(n - 3, n)[None], th, m)
    bound = 8 * 2.0 ** -24 * _pair_sum(_np(last), d, False) + 2.0 ** -20 * _pair_sum(_np(last), d, False)
    _close(x[:, -3:], ref, bound + 2.0 ** -8 * (np.abs(ref) + bound), "rope")
    assert not x[:, :-3].any()


def test_tree_on_a_stream_of_its_own_keeps_its_memory():
    # What the call allocates for another stream is that stream's: neither a block that the current stream
    # still writes, nor, freed on return, one that it may write next while the other still computes.
    B, T, H, d, n = 1, 8, 8, 64, 200000
    g = _gen(8)
    c = da.cache_v1(B, n, H, d)
    for t in (c.k1, c.k2, c.v):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
    q1, q2, lam = _bf(g, B, T, H, d), _bf(g, B, T, H, d), torch.tensor([0.4], device="cuda")
    ref = da.tree_decode(q1, q2, c, lam, 0.3)
    need = da.tree_decode_workspace_bytes(B, T, H, d)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        a, b = torch.empty_like(ref), torch.empty(need, dtype=torch.uint8, device="cuda")
        torch.cuda._sleep(2000000)
        a.fill_(float("nan"))
        b.fill_(255)
        del a, b
        out = da.tree_decode(q1, q2, c, lam, 0.3, stream=s)
        torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    da.device_status()


def test_step_replays_in_a_graph_and_on_two_streams():
    # One speculative step captured and replayed on new inputs: the eager call's bits; and two such
    # steps at once on two streams, with caches of their own.
    B, H, d, T, n = 3, 4, 128, 9, 700
    g = _gen(31)
    spec = da.rope_spec(d, scaling="yarn", factor=4.0, original_context=512)
    rs = np.random.RandomState(3)
    mask = [_tree_mask(rs, T) for _ in range(B)]

    def state(fmt):
        c, _, _ = _random_cache(g, B, n, H, d, True, fmt)
        st = {"pos": None, "lens": _i32([600, 0, 77]), "ntok": _i32([9, 4, 7]), "mask": _words(mask),
              "lam": torch.tensor([0.4], device="cuda"), "path": _i32([[0, 3, 4, 8] + [0] * 5] * B),
              "nkeep": _i32([4, 1, 3])}
        return c, st
    for fmt in ("bf16", "fp8"):
        c, st = state(fmt)
        x = _speculative(g, B, T, H, d)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            _step(c, x, st, spec, T)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got, new = _step(c, x, st, spec, T)
        start = _contents(c)
        for _ in range(2):
            for t in x.values():
                t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
            for t, o in zip((c.k1, c.k2, c.v, c.k1_scales, c.k2_scales, c.v_scales), start + [None] * 3):
                if o is not None:
                    t.copy_(o)
            graph.replay()
            torch.cuda.synchronize()
            da.device_status()
            after = _contents(c)
            for t, o in zip((c.k1, c.k2, c.v, c.k1_scales, c.k2_scales, c.v_scales), start + [None] * 3):
                if o is not None:
                    t.copy_(o)
            want, wnew = _step(c, x, st, spec, T)
            da.device_status()
            assert torch.equal(got, want) and torch.equal(new, wnew) and _same(after, _contents(c))
    two = [state("fp8") for _ in range(2)]
    xs = [_speculative(g, B, T, H, d) for _ in range(2)]
    start = [_contents(c) for c, _ in two]
    alone = [_step(c, x, st, spec, T)[0] for (c, st), x in zip(two, xs)]
    da.device_status()
    for (c, _), old in zip(two, start):
        for t, o in zip((c.k1, c.k2, c.v, c.k1_scales, c.k2_scales, c.v_scales), old):
            t.copy_(o)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    both = []
    for (c, st), x, s in zip(two, xs, streams):
        with torch.cuda.stream(s):
            both.append(_step(c, x, st, spec, T)[0])
    torch.cuda.synchronize()
    da.device_status()
    assert all(torch.equal(a, b) for a, b in zip(alone, both))
