"""Rotary positions, caches and draft trees without a GPU: the fp64 references' pins, the host-side
rotary tables, and every refusal of the C entry points and the binding (nothing is launched)."""

import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
from differential_attention_03_gb300 import binding as da
from differential_attention_03_gb300 import build


@pytest.fixture(scope="module")
def L():
    build.build()
    return da.lib()


P = ctypes.c_void_p
A, A2, A3 = P(0x10000), P(0x4000000), P(0x8000000)  # aligned fake device addresses, never dereferenced
MIS = P(0x10008)


# ----------------------------------------------------------------------------- references
def test_reference_rotation_keeps_relative_positions():
    rs = np.random.RandomState(0)
    th, _ = oracle.rope_frequencies(16)
    q, k = rs.randn(1, 1, 1, 16), rs.randn(1, 1, 1, 16)
    for inter in (False, True):
        def dot(a, b):
            return (oracle.rope(q, [[a]], th, 1.0, inter) * oracle.rope(k, [[b]], th, 1.0, inter)).sum()
        assert dot(5, 3) == pytest.approx(dot(1002, 1000), rel=1e-9)
        x = oracle.rope(q, [[7]], th, 1.3, inter)
        assert np.allclose(oracle.rope(x, [[7]], th, 1.3, inter, inverse=True), 1.69 * q)


def test_reference_e4m3_rounding_agrees_with_torch():
    x = np.concatenate([np.random.RandomState(1).randn(4000) * s for s in (0.01, 1, 100)] + [np.array([0, 464, 1e9, -1e9])])
    t = torch.tensor(x, dtype=torch.float32).clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.e4m3_round(x.astype(np.float32)), t)


def test_reference_chain_is_the_causal_forward():
    rs = np.random.RandomState(2)
    B, n, T, H, d = 2, 9, 4, 2, 8
    q1, q2, k1, k2 = (rs.randn(B, n, H, d) for _ in range(4))
    v = rs.randn(B, n, H, 2 * d)
    gamma = rs.rand(2 * d)
    ref = oracle.diff_attn_v1(q1, q2, k1, k2, v, 0.4, 0.3, gamma, 1e-5, True)
    got = oracle.tree_v1(q1[:, n - T:], q2[:, n - T:], k1, k2, v, [n - T] * B, [T] * B, None, 0.4, 0.3, gamma, 1e-5)[0]
    assert np.allclose(got, ref[:, n - T:])
    q, k, v = rs.randn(B, n, 4, d), rs.randn(B, n, 2, d), rs.randn(B, n, 2, d)
    lg = rs.randn(B, n, 2)
    ref = oracle.diff_attn_v2(q, k, v, lg, True)
    got = oracle.tree_v2(q[:, n - T:], k, v, lg[:, n - T:], [n - T] * B, [T] * B, None)[0]
    assert np.allclose(got, ref[:, n - T:])


# ----------------------------------------------------------------------------- rotary tables
@pytest.mark.parametrize("rot,base,inter,scaling,factor,orig", [
    (64, 10000.0, False, "none", 1.0, 0), (128, 500000.0, True, "linear", 8.0, 0), (4, 10000.0, False, "ntk", 4.0, 0),
    (128, 10000.0, False, "yarn", 32.0, 4096), (2, 100.0, True, "none", 1.0, 0), (26, 10000.0, False, "yarn", 2.0, 100)])
def test_rope_table_holds_the_frequencies(L, rot, base, inter, scaling, factor, orig):
    spec = da.rope_spec(rot, base, inter, scaling, factor, orig)
    th, m = oracle.rope_frequencies(rot, base, scaling, factor, orig)
    assert (spec.rot_dim, spec.interleaved, spec.mult) == (rot, int(inter), np.float32(m))
    for i in range(rot // 2):
        assert spec.turns[i] / 2.0 ** 64 == pytest.approx(th[i] / (2 * math.pi), rel=1e-14, abs=2.0 ** -62)
    assert da.rope_spec(rot, base, inter, scaling, factor, orig) is spec
    own = da.rope_from_frequencies(th, inter, m)
    assert list(own.turns)[:rot // 2] == pytest.approx(list(spec.turns)[:rot // 2], rel=1e-14)


def test_rope_table_takes_any_finite_frequency(L):
    s = da.rope_from_frequencies([2 * math.pi, -1.0, 100.0, -1e-300])
    assert s.turns[0] == 0 and s.turns[3] == 0
    assert s.turns[1] / 2.0 ** 64 == pytest.approx(1 - 1 / (2 * math.pi))
    assert s.turns[2] / 2.0 ** 64 == pytest.approx((100 / (2 * math.pi)) % 1)


@pytest.mark.parametrize("args,status", [
    ((0,), da.ERR_SHAPE), ((3,), da.ERR_SHAPE), ((130,), da.ERR_SHAPE), ((64, 1.0), da.ERR_SHAPE),
    ((64, float("inf")), da.ERR_SHAPE), ((64, 1e4, False, "linear", 0.5), da.ERR_SHAPE),
    ((64, 1e4, False, "linear", float("nan")), da.ERR_SHAPE), ((2, 1e4, False, "ntk", 2.0), da.ERR_SHAPE),
    ((64, 1e4, False, "yarn", 2.0, 0), da.ERR_SHAPE), ((64, 1e4, False, "yarn", 2.0, 100, 0.0), da.ERR_SHAPE)])
def test_rope_table_refusals(L, args, status):
    with pytest.raises(da.DiffAttnError) as e:
        da.rope_spec(*args)
    assert e.value.status == status


def test_rope_table_refusals_of_the_abi(L):
    d = ctypes.c_double
    spec = da.RopeSpec()
    assert L.diffattn_rope_init(None, 64, 0, d(1e4), 0, d(1), 0, d(32), d(1)) == da.ERR_NULL
    assert L.diffattn_rope_init(ctypes.byref(spec), 64, 0, d(1e4), 9, d(1), 0, d(32), d(1)) == da.ERR_DTYPE
    f = (d * 2)(1.0, float("inf"))
    assert L.diffattn_rope_from_frequencies(ctypes.byref(spec), 4, 0, f, ctypes.c_float(1)) == da.ERR_SHAPE
    assert L.diffattn_rope_from_frequencies(ctypes.byref(spec), 4, 0, None, ctypes.c_float(1)) == da.ERR_NULL
    f = (d * 2)(1.0, 2.0)
    assert L.diffattn_rope_from_frequencies(ctypes.byref(spec), 4, 0, f, ctypes.c_float(float("nan"))) == da.ERR_SHAPE
    with pytest.raises(ValueError):
        da.rope_spec(64, scaling="other")


# ----------------------------------------------------------------------------- refusals
def _rope(L, dt=1, B=1, n=4, d=64, xs=(A,), heads=(2,), spec="ok", out=(A2,), rot=64, count=None):
    s = da.rope_spec(rot) if spec == "ok" else spec
    m = len(xs)
    return L.diffattn_rope(dt, B, n, d, m if count is None else count, (P * m)(*[x.value if x else None for x in xs]),
                           (ctypes.c_int * m)(*heads), None if s is None else ctypes.byref(s), None, 0,
                           (P * m)(*[o.value if o else None for o in out]), None)


def test_rope_refusals(L):
    assert _rope(L, dt=5) == da.ERR_DTYPE
    assert _rope(L, B=-1) == da.ERR_SHAPE
    assert _rope(L, d=0) == da.ERR_SHAPE
    assert _rope(L, B=0) == da.OK and _rope(L, n=0) == da.OK and _rope(L, count=0) == da.OK
    assert _rope(L, count=5) == da.ERR_UNSUPPORTED
    assert _rope(L, d=256) == da.ERR_UNSUPPORTED
    assert _rope(L, d=32) == da.ERR_SHAPE  # fewer channels than are rotated
    assert _rope(L, spec=None) == da.ERR_NULL
    assert _rope(L, xs=(None,)) == da.ERR_NULL
    assert _rope(L, out=(None,)) == da.ERR_NULL
    assert _rope(L, heads=(-1,)) == da.ERR_SHAPE
    assert _rope(L, heads=(0,), xs=(None,), out=(None,)) == da.OK
    assert _rope(L, xs=(MIS,)) == da.ERR_ALIGN
    assert _rope(L, out=(P(0x10100),)) == da.ERR_SHAPE                        # half over its input
    assert _rope(L, xs=(A, A2), heads=(1, 1), out=(A2, A3)) == da.ERR_SHAPE    # over another's input
    assert _rope(L, xs=(A, A2), heads=(1, 1), out=(A3, A3)) == da.ERR_SHAPE
    bad = da.RopeSpec.from_buffer_copy(da.rope_spec(64))
    bad.mult = float("inf")
    assert _rope(L, spec=bad) == da.ERR_SHAPE
    bad.mult, bad.rot_dim = 1.0, 7
    assert _rope(L, spec=bad) == da.ERR_SHAPE


def _append(L, fmt=0, B=1, T=2, H=1, n=8, d=64, q=(A, A), k=(A, A), v=A, qo=(A2, A3), kc=(A, A), vc=A, ks=(1.0, 1.0),
            sc=(A, A, A), spec=None):
    f = ctypes.c_float
    return L.diffattn_cache_append(fmt, B, T, H, n, d, *q, *k, v, None if spec is None else ctypes.byref(spec), None,
                                   None, None, *qo, *kc, vc, f(ks[0]), f(ks[1]), *sc, None)


def test_append_refusals(L):
    assert _append(L, fmt=3) == da.ERR_DTYPE
    assert _append(L, T=-1) == da.ERR_SHAPE
    assert _append(L, B=0) == da.OK and _append(L, T=0) == da.OK
    assert _append(L, d=96) == da.ERR_UNSUPPORTED
    assert _append(L, k=(A, None)) == da.ERR_NULL
    assert _append(L, v=None) == da.ERR_NULL
    assert _append(L, vc=None) == da.ERR_NULL
    assert _append(L, q=(A, None)) == da.ERR_NULL
    assert _append(L, qo=(A2, None)) == da.ERR_NULL
    assert _append(L, k=(A, MIS)) == da.ERR_ALIGN
    assert _append(L, qo=(A2, P(0x8000008))) == da.ERR_ALIGN
    assert _append(L, qo=(A, A2)) == da.ERR_SHAPE
    assert _append(L, fmt=1, ks=(0.0, 1.0)) == da.ERR_SHAPE
    assert _append(L, fmt=1, ks=(1.0, float("nan"))) == da.ERR_SHAPE
    assert _append(L, fmt=2, sc=(A, None, A)) == da.ERR_NULL
    assert _append(L, fmt=2, sc=(A, A, None)) == da.ERR_NULL
    assert _append(L, fmt=2, sc=(A, P(0x10002), A)) == da.ERR_ALIGN
    assert _append(L, spec=da.rope_spec(128)) == da.ERR_SHAPE
    f = ctypes.c_float
    v2 = lambda d=128, q=A: L.diffattn_v2_cache_append(0, 1, 2, 4, 2, 8, d, q, A, A, None, None, None, None, A2, A, A,  # noqa: E731
                                                       f(1), None, None, None)
    assert v2(d=64) == da.ERR_UNSUPPORTED
    assert v2(q=A2) == da.ERR_SHAPE


def test_append_refuses_overlaps(L):
    # distinct tensors of 64 KB each but for one: what is written meets an input, or another output
    at = [P(0x100000 * (i + 1)) for i in range(13)]
    full = dict(fmt=2, q=(at[0], at[1]), k=(at[2], at[3]), v=at[4], qo=(at[5], at[6]), kc=(at[7], at[8]), vc=at[9],
                sc=(at[10], at[11], at[12]))

    def with_(**kw):
        status = _append(L, **{**full, **kw})
        return status, L.diffattn_last_error()
    for kw in (dict(qo=(at[0], at[6])), dict(qo=(at[5], at[0])), dict(qo=(at[2], at[6])), dict(qo=(at[5], at[5])),
               dict(qo=(at[7], at[6])), dict(kc=(at[2], at[8])), dict(kc=(at[7], at[7])), dict(kc=(at[7], at[4])),
               dict(vc=at[4]), dict(vc=at[8]), dict(sc=(at[10], at[10], at[12])), dict(sc=(at[10], at[11], at[9])),
               dict(vc=P(at[4].value + 16)), dict(sc=(at[3], at[11], at[12]))):
        status, why = with_(**kw)
        assert status == da.ERR_SHAPE and b"overlap" in why, kw


def test_keep_refuses_overlaps(L):
    a, b = P(0x100000), P(0x200000)
    for tensors in ((a, a, b), (a, b, a), (a, b, P(0x200000 + 512))):
        assert L.diffattn_cache_keep(0, 1, 2, 1, 8, 64, *tensors, None, None, None, A, A2, A3, None, None) == da.ERR_SHAPE
        assert b"overlap" in L.diffattn_last_error()


def _tree(L, fmt=0, B=1, T=2, H=1, n=8, d=64, q=(A, A), k=(A, A), v=A, ks=(1.0, 1.0), sc=(A, A, A), mask=None, sb=0,
          lam=A, lin=0.2, out=A, ws=A, wn=1 << 30):
    f = ctypes.c_float
    return L.diffattn_tree_decode(fmt, B, T, H, n, d, *q, *k, f(ks[0]), f(ks[1]), sc[0], sc[1], v, sc[2], None, None,
                                  mask, sb, lam, f(lin), None, f(1e-5), out, ws, wn, None)


def test_tree_refusals(L):
    assert _tree(L, fmt=-1) == da.ERR_DTYPE
    assert _tree(L, n=-1) == da.ERR_SHAPE
    assert _tree(L, sb=-1) == da.ERR_SHAPE
    assert _tree(L, B=0) == da.OK and _tree(L, T=0) == da.OK and _tree(L, H=0) == da.OK
    assert _tree(L, T=65) == da.ERR_UNSUPPORTED
    assert _tree(L, d=32) == da.ERR_UNSUPPORTED
    assert _tree(L, q=(A, None)) == da.ERR_NULL
    assert _tree(L, lam=None) == da.ERR_NULL
    assert _tree(L, lin=float("inf")) == da.ERR_SHAPE
    assert _tree(L, ws=None) == da.ERR_NULL
    assert _tree(L, wn=16) == da.ERR_SHAPE
    assert _tree(L, ws=MIS) == da.ERR_ALIGN
    assert _tree(L, out=MIS) == da.ERR_ALIGN
    assert _tree(L, mask=P(0x10004)) == da.ERR_ALIGN
    assert _tree(L, fmt=1, ks=(1.0, -1.0)) == da.ERR_SHAPE
    assert _tree(L, fmt=2, sc=(None, A, A)) == da.ERR_NULL
    assert _tree(L, B=1 << 20, H=1 << 10) == da.ERR_SHAPE
    f = ctypes.c_float

    def v2(Hq=4, Hkv=2, d=128, logits=A, scale=0.0):
        return L.diffattn_v2_tree_decode(0, 1, 2, Hq, Hkv, 8, d, A, A, f(1), None, A, None, None, None, None, 0, logits,
                                         0, 0, f(scale), A, A, 1 << 30, None)
    assert v2(Hq=6, Hkv=2) == da.ERR_SHAPE
    assert v2(Hkv=0) == da.ERR_SHAPE
    assert v2(d=64) == da.ERR_UNSUPPORTED
    assert v2(logits=None) == da.ERR_NULL
    assert v2(scale=float("inf")) == da.ERR_SHAPE
    assert b"softmax_scale" in L.diffattn_last_error()


def test_tree_workspace_sizes(L):
    # a partial state of 2 R (dv + 2) floats a row tile and a CTA; four of them up to 8 rows, two up to 32
    # (O from a multiple of 8 floats on; 16 bytes to reach a 32-byte boundary)
    assert da.tree_decode_workspace_bytes(2, 5, 3, 64) == (6 + 160) * 4 * 2 * 5 * 130 * 4 + 16
    assert da.tree_decode_workspace_bytes(2, 9, 3, 128) == (6 + 160) * 2 * 2 * 9 * 258 * 4 + 16
    assert da.v2_tree_decode_workspace_bytes(1, 20, 16, 2, 128) == (1 * 2 * 2 + 160) * 2 * 60 * 130 * 4 + 16
    assert da.v2_tree_decode_workspace_bytes(1, 64, 8, 1, 128) == (4 + 160) * 2 * 64 * 130 * 4 + 16
    assert da.tree_decode_workspace_bytes(1, 65, 1, 64) == 0
    assert da.v2_tree_decode_workspace_bytes(1, 4, 6, 2, 128) == 0


def _keep(L, fmt=0, B=1, n=8, d=64, a=4, k=(A, A), v=A, sc=(A, A, A), lens=A, path=A, nkeep=A, new=A2):
    return L.diffattn_cache_keep(fmt, B, a, 2, n, d, *k, v, *sc, lens, path, nkeep, new, None)


def test_keep_refusals(L):
    assert _keep(L, fmt=4) == da.ERR_DTYPE
    assert _keep(L, a=-1) == da.ERR_SHAPE
    assert _keep(L, a=65) == da.ERR_UNSUPPORTED
    assert _keep(L, B=0) == da.OK
    assert _keep(L, d=63) == da.ERR_UNSUPPORTED
    for name in ("lens", "path", "nkeep", "v"):
        assert _keep(L, **{name: None}) == da.ERR_NULL
    assert _keep(L, k=(A, None)) == da.ERR_NULL
    assert _keep(L, k=(A, MIS)) == da.ERR_ALIGN
    assert _keep(L, new=A) == da.ERR_SHAPE  # lens itself
    assert _keep(L, fmt=2, sc=(A, A, None)) == da.ERR_NULL
    assert L.diffattn_v2_cache_keep(0, 1, 4, 2, 8, 64, A, A, None, None, A, A, A, A2, None) == da.ERR_UNSUPPORTED


def test_binding_refuses_tensors_off_the_gpu(L):
    x = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        da.rope([x], da.rope_spec(64))
    with pytest.raises(ValueError):
        da.KVCache("bf16", x, x, x)
    with pytest.raises(ValueError):
        da.KVCache("int4", x, x, x)
    with pytest.raises(ValueError):
        da.cache_v1(1, 2, 1, 64, "int4", device="cpu")
    with pytest.raises(ValueError):
        da.rope([x] * 5, da.rope_spec(64))
    assert da.rope([], da.rope_spec(64)) == []
