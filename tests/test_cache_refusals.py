"""Calls of the cache operators that are refused on the host (fake addresses: nothing is launched)."""

import ctypes

import pytest

from differential_attention_03_gb300 import binding as da
from differential_attention_03_gb300 import build


@pytest.fixture(scope="module")
def L():
    build.build()
    return da.lib()


P = ctypes.c_void_p
AT = [P(0x100000 * (i + 1)) for i in range(24)]  # 1 MB apart; the tensors here are smaller


def _overlap(L, status):
    return status == da.ERR_SHAPE and b"overlap" in L.diffattn_last_error()


def _keep(L, fmt=2, k=(AT[0], AT[1]), v=AT[2], sc=(AT[3], AT[4], AT[5]), lens=AT[6], path=AT[7], nkeep=AT[8],
          new=AT[9]):
    return L.diffattn_cache_keep(fmt, 4, 8, 2, 64, 64, *k, v, *sc, lens, path, nkeep, new, None)


def test_keep_refuses_what_it_writes_over_what_it_reads(L):
    # new_lens is written by one CTA of a sequence while others still read nkeep and path
    for kw in (dict(new=AT[8]), dict(new=P(AT[8].value + 12)), dict(new=AT[7]), dict(new=P(AT[7].value + 4 * 31)),
               dict(new=AT[6]), dict(new=AT[1]), dict(new=P(AT[2].value + 128)), dict(new=AT[5]),
               dict(sc=(AT[3], AT[3], AT[5])), dict(sc=(AT[3], AT[4], AT[4])), dict(sc=(AT[0], AT[4], AT[5])),
               dict(sc=(AT[3], AT[4], P(AT[2].value + 64))), dict(path=AT[0]), dict(lens=AT[4]), dict(nkeep=AT[2])):
        assert _overlap(L, _keep(L, **kw)), kw
    for kw in (dict(new=AT[8]), dict(k=(AT[0], AT[0]))):
        assert _overlap(L, _keep(L, fmt=0, sc=(None, None, None), **kw)), kw
    assert _overlap(L, L.diffattn_v2_cache_keep(2, 4, 8, 2, 64, 128, AT[0], AT[1], AT[2], AT[2], AT[6], AT[7], AT[8],
                                                AT[9], None))


def _append(L, fmt=2, q=(AT[0], AT[1]), k=(AT[2], AT[3]), v=AT[4], pos=AT[5], lens=AT[6], ntok=AT[7], qo=(AT[8], AT[9]),
            kc=(AT[10], AT[11]), vc=AT[12], sc=(AT[13], AT[14], AT[15]), scale=1.0):
    f = ctypes.c_float
    return L.diffattn_cache_append(fmt, 4, 8, 2, 64, 64, *q, *k, v, None, pos, lens, ntok, *qo, *kc, vc, f(scale),
                                   f(scale), *sc, None)


def test_append_refuses_outputs_over_its_index_tensors(L):
    for name in ("pos", "lens", "ntok"):
        for at in (AT[8], AT[9], AT[10], AT[11], AT[12], AT[13], AT[15], P(AT[8].value + 64)):
            assert _overlap(L, _append(L, **{name: at})), (name, at)


def test_rope_refuses_an_output_over_the_positions(L):
    spec = da.rope_spec(64)
    for pos in (AT[1], P(AT[1].value + 256), AT[0]):
        xs, outs = (P * 2)(AT[0].value, AT[3].value), (P * 2)(AT[0].value, AT[1].value)
        assert _overlap(L, L.diffattn_rope(1, 2, 8, 64, 2, xs, (ctypes.c_int * 2)(2, 2), ctypes.byref(spec), pos, 0, outs,
                                           None)), pos


def _tree(L, fmt=2, q=(AT[0], AT[1]), k=(AT[2], AT[3]), v=AT[4], sc=(AT[5], AT[6], AT[7]), lens=AT[8], ntok=AT[9],
          mask=AT[10], sb=4, lam=AT[11], gamma=AT[12], out=AT[13], ws=P(0x10000000)):
    f = ctypes.c_float
    return L.diffattn_tree_decode(fmt, 4, 4, 2, 64, 64, *q, *k, f(1), f(1), sc[0], sc[1], v, sc[2], lens, ntok, mask, sb,
                                  lam, f(0.2), gamma, f(1e-5), out, ws, 1 << 30, None)


def test_tree_refuses_outputs_over_what_it_reads(L):
    for at in AT[2:13]:
        assert _overlap(L, _tree(L, out=at)), at
    for at in AT[:14]:
        assert _overlap(L, _tree(L, ws=at)), at
    assert _overlap(L, _tree(L, out=P(0x10000000 + 4096)))
    assert _overlap(L, _tree(L, out=P(AT[10].value + 96)))  # (the last sequence's mask words)
    f = ctypes.c_float

    def v2(out=AT[5], ws=P(0x10000000), logits=AT[4]):
        return L.diffattn_v2_tree_decode(0, 2, 4, 8, 2, 64, 128, AT[0], AT[1], f(1), None, AT[2], None, None, None, None, 0,
                                         logits, 16, 4, f(0), out, ws, 1 << 30, None)
    for kw in (dict(out=AT[1]), dict(out=AT[2]), dict(out=AT[4]), dict(out=P(AT[4].value + 112)), dict(ws=AT[0]),
               dict(ws=AT[4]), dict(ws=AT[2])):
        assert _overlap(L, v2(**kw)), kw


def test_a_key_scale_without_a_reciprocal_is_refused(L):
    # keys are multiplied by 1 / scale: an infinity would make a zero key NaN
    for scale in (2.0 ** -129, 1e-45):
        assert _append(L, fmt=1, scale=scale) == da.ERR_SHAPE, scale
        assert b"reciprocal" in L.diffattn_last_error()


def test_append_refuses_queries_without_a_key_head(L):
    f = ctypes.c_float

    def v2(Hq, q):
        return L.diffattn_v2_cache_append(0, 1, 2, Hq, 0, 8, 128, q, None, None, None, None, None, None, AT[1], None, None,
                                          f(1), None, None, None)
    assert v2(4, AT[0]) == da.ERR_SHAPE and b"key head" in L.diffattn_last_error()
    assert v2(4, None) == da.OK and v2(0, AT[0]) == da.OK


def test_a_shared_rotation_cannot_be_changed(L):
    spec = da.rope_spec(64, base=777.0)
    before = bytes(spec)
    for name, x in (("mult", 2.0), ("rot_dim", 2), ("interleaved", 1), ("turns", (ctypes.c_ulonglong * 64)())):
        with pytest.raises(AttributeError):
            setattr(spec, name, x)
    spec.turns[1] = 5  # (a copy's)
    assert da.rope_spec(64, base=777.0) is spec and bytes(spec) == before
    own = da.RopeSpec.from_buffer_copy(spec)
    own.mult, own.turns[1] = 2.0, 5
    assert (own.mult, own.turns[1]) == (2.0, 5) and bytes(spec) == before
