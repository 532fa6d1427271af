"""Calls of the block's operators that are refused on the host, and sizes of their workspaces (fake addresses: nothing is
launched)."""

import ctypes

import pytest
import torch

from differential_attention_03_gb300 import binding as da
from differential_attention_03_gb300 import build


@pytest.fixture(scope="module")
def L():
    build.build()
    return da.lib()


P = ctypes.c_void_p
AT = [P(0x1000000 * (i + 1)) for i in range(24)]  # 16 MB apart; the tensors here are smaller
WS, ROOM = P(0x70000000), 1 << 30
F = ctypes.c_float


def _off(p, n):
    return P(p.value + n)


def _linear(L, M=64, N=256, K=128, a=AT[0], lda=128, w=AT[1], bias=AT[2], act=2, res=AT[3], ldr=256, dt=1, out=AT[4], ldo=256,
            pre=AT[5]):
    return L.diffattn_linear(M, N, K, a, lda, w, bias, act, res, ldr, dt, out, ldo, pre, None)


def test_linear_refuses(L):
    for kw, want in ((dict(M=-1), da.ERR_SHAPE), (dict(N=-8), da.ERR_SHAPE), (dict(K=0), da.ERR_SHAPE),
                     (dict(K=124, lda=128), da.ERR_SHAPE), (dict(N=252), da.ERR_SHAPE), (dict(act=5), da.ERR_DTYPE),
                     (dict(act=-1), da.ERR_DTYPE), (dict(dt=2), da.ERR_DTYPE), (dict(a=None), da.ERR_NULL),
                     (dict(w=None), da.ERR_NULL), (dict(out=None), da.ERR_NULL), (dict(lda=120), da.ERR_SHAPE),
                     (dict(lda=132), da.ERR_SHAPE), (dict(ldo=248), da.ERR_SHAPE), (dict(ldo=260), da.ERR_SHAPE),
                     (dict(ldr=128), da.ERR_SHAPE), (dict(a=_off(AT[0], 8)), da.ERR_ALIGN), (dict(w=_off(AT[1], 2)), da.ERR_ALIGN),
                     (dict(out=_off(AT[4], 8)), da.ERR_ALIGN), (dict(res=_off(AT[3], 8)), da.ERR_ALIGN),
                     (dict(bias=_off(AT[2], 4)), da.ERR_ALIGN), (dict(pre=_off(AT[5], 8)), da.ERR_ALIGN),
                     (dict(M=0x7fffff80, lda=128), da.ERR_SHAPE), (dict(dt=0, ldo=258), da.ERR_SHAPE)):
        assert _linear(L, **kw) == want, kw
    assert _linear(L, M=0, a=None, out=None) == da.OK and _linear(L, N=0, w=None, out=None) == da.OK


def test_linear_refuses_overlap(L):
    def over(**kw):
        return _linear(L, **kw) == da.ERR_SHAPE and b"overlap" in L.diffattn_last_error()
    for kw in (dict(out=AT[0]), dict(out=AT[1]), dict(out=AT[2]), dict(pre=AT[4]), dict(pre=AT[3]), dict(pre=AT[0]),
               dict(out=_off(AT[3], 16)), dict(out=AT[3], ldr=256, ldo=264), dict(out=_off(AT[0], 64 * 256 - 32)),
               # rows side by side that reach into each other
               dict(a=AT[0], lda=512, out=_off(AT[0], 128 * 2 - 16), ldo=512),
               dict(a=_off(AT[0], 512), lda=512, out=AT[0], ldo=384, res=None),
               dict(res=AT[4], out=AT[4], pre=AT[4])):
        assert over(**kw), kw


def test_rows_side_by_side_are_no_overlap(L):
    # (the calls go on to refuse a later fault, so that nothing is launched)
    status = _linear(L, a=AT[0], lda=512, out=_off(AT[0], 256), ldo=512, res=None, pre=AT[0], bias=None)
    assert status == da.ERR_SHAPE and b"overlap" in L.diffattn_last_error()  # pre over a, not out beside it
    status = _linear(L, res=_off(AT[4], 512), ldr=512, out=AT[4], ldo=512, pre=AT[0], bias=None)
    assert status == da.ERR_SHAPE and b"input" in L.diffattn_last_error()


def _linear_bwd(L, M=64, N=256, K=128, a=AT[0], lda=128, w=AT[1], dy=AT[2], ldy=256, pre=AT[3], act=4, dx=AT[4], dw=AT[5], dt=0,
                db=AT[6], ws=WS, room=ROOM):
    return L.diffattn_linear_backward(M, N, K, a, lda, w, dy, ldy, pre, act, dx, dw, dt, db, ws, room, None)


def test_linear_backward_refuses(L):
    need = L.diffattn_linear_backward_workspace(64, 256, 128)
    for kw, want in ((dict(K=0), da.ERR_SHAPE), (dict(N=250), da.ERR_SHAPE), (dict(act=9), da.ERR_DTYPE), (dict(dt=3), da.ERR_DTYPE),
                     (dict(a=None), da.ERR_NULL), (dict(w=None), da.ERR_NULL), (dict(dy=None), da.ERR_NULL),
                     (dict(pre=None), da.ERR_NULL), (dict(ws=None), da.ERR_NULL), (dict(room=need - 1), da.ERR_SHAPE),
                     (dict(ws=_off(WS, 16)), da.ERR_ALIGN), (dict(ldy=255), da.ERR_SHAPE), (dict(lda=136 + 4), da.ERR_SHAPE),
                     (dict(dx=_off(AT[4], 8)), da.ERR_ALIGN), (dict(dw=_off(AT[5], 8)), da.ERR_ALIGN),
                     (dict(db=_off(AT[6], 2)), da.ERR_ALIGN), (dict(dx=AT[2]), da.ERR_SHAPE), (dict(dw=AT[0]), da.ERR_SHAPE),
                     (dict(db=AT[3]), da.ERR_SHAPE), (dict(dw=AT[4]), da.ERR_SHAPE), (dict(ws=AT[2]), da.ERR_SHAPE),
                     (dict(dx=_off(WS, 256)), da.ERR_SHAPE)):
        assert _linear_bwd(L, **kw) == want, kw
    assert _linear_bwd(L, dx=None, dw=None, db=None) == da.OK  # nothing asked for


def _gated(L, M=64, D=128, F=256, x=AT[0], ldx=128, w=AT[1], act=4, h=AT[2], ldh=256, gu=AT[3]):
    return L.diffattn_gated_linear(M, D, F, x, ldx, w, act, h, ldh, gu, None)


def test_gated_refuses(L):
    for kw, want in ((dict(D=0), da.ERR_SHAPE), (dict(D=100, ldx=104), da.ERR_SHAPE), (dict(F=252), da.ERR_SHAPE), (dict(M=-1), da.ERR_SHAPE),
                     (dict(act=7), da.ERR_DTYPE), (dict(x=None), da.ERR_NULL), (dict(w=None), da.ERR_NULL), (dict(h=None), da.ERR_NULL),
                     (dict(ldx=64), da.ERR_SHAPE), (dict(ldh=255), da.ERR_SHAPE), (dict(h=_off(AT[2], 8)), da.ERR_ALIGN),
                     (dict(gu=_off(AT[3], 8)), da.ERR_ALIGN), (dict(h=AT[0]), da.ERR_SHAPE), (dict(gu=AT[1]), da.ERR_SHAPE),
                     (dict(h=_off(AT[1], 511 * 256)), da.ERR_SHAPE), (dict(gu=AT[2]), da.ERR_SHAPE), (dict(F=0x40000000), da.ERR_SHAPE)):
        assert _gated(L, **kw) == want, kw
    assert _gated(L, M=0, x=None) == da.OK and _gated(L, F=0, w=None) == da.OK


def _gated_bwd(L, M=64, D=128, F=256, x=AT[0], ldx=128, w=AT[1], gu=AT[2], dh=AT[3], ldh=256, act=4, dx=AT[4], dw=AT[5], dt=1, ws=WS,
               room=ROOM):
    return L.diffattn_gated_linear_backward(M, D, F, x, ldx, w, gu, dh, ldh, act, dx, dw, dt, ws, room, None)


def test_gated_backward_refuses(L):
    need = L.diffattn_gated_linear_backward_workspace(64, 128, 256)
    assert need >= 64 * 512 * 2
    for kw, want in ((dict(act=5), da.ERR_DTYPE), (dict(dt=2), da.ERR_DTYPE), (dict(gu=None), da.ERR_NULL), (dict(dh=None), da.ERR_NULL),
                     (dict(x=None), da.ERR_NULL), (dict(w=None), da.ERR_NULL), (dict(ws=None), da.ERR_NULL),
                     (dict(room=need - 1), da.ERR_SHAPE), (dict(ldh=128), da.ERR_SHAPE), (dict(dx=AT[3]), da.ERR_SHAPE),
                     (dict(dw=AT[2]), da.ERR_SHAPE), (dict(dw=AT[4]), da.ERR_SHAPE), (dict(ws=AT[2]), da.ERR_SHAPE)):
        assert _gated_bwd(L, **kw) == want, kw
    assert _gated_bwd(L, dx=None, dw=None, gu=None) == da.OK


def _norm(L, dt=1, sdt=0, rows=12, D=256, x=AT[0], res=AT[1], gate=AT[2], G=3, scale=1.0, post=1, gp=AT[3], ga=AT[4], eps=1e-5,
          s=AT[5], y=AT[6]):
    return L.diffattn_residual_norm(dt, sdt, rows, D, x, res, gate, G, F(scale), post, gp, ga, F(eps), s, y, None)


def test_norm_refuses(L):
    nan = float("nan")
    for kw, want in ((dict(dt=0, sdt=1), da.ERR_DTYPE), (dict(dt=2), da.ERR_DTYPE), (dict(rows=-1), da.ERR_SHAPE), (dict(D=0), da.ERR_SHAPE),
                     (dict(D=8193), da.ERR_UNSUPPORTED), (dict(G=0), da.ERR_SHAPE), (dict(G=5), da.ERR_SHAPE), (dict(G=24), da.ERR_SHAPE),
                     (dict(scale=nan), da.ERR_SHAPE), (dict(scale=float("inf")), da.ERR_SHAPE), (dict(post=0), da.ERR_SHAPE),
                     (dict(s=None, y=None, ga=None), da.ERR_SHAPE), (dict(y=None), da.ERR_SHAPE), (dict(x=None), da.ERR_NULL),
                     (dict(x=_off(AT[0], 8)), da.ERR_ALIGN), (dict(s=_off(AT[5], 4)), da.ERR_ALIGN), (dict(gate=_off(AT[2], 4)), da.ERR_ALIGN),
                     (dict(s=AT[0]), da.ERR_SHAPE), (dict(y=AT[0]), da.ERR_SHAPE), (dict(y=AT[1]), da.ERR_SHAPE), (dict(y=AT[5]), da.ERR_SHAPE),
                     (dict(s=_off(AT[1], 1024)), da.ERR_SHAPE), (dict(s=AT[2]), da.ERR_SHAPE), (dict(y=AT[4]), da.ERR_SHAPE)):
        assert _norm(L, **kw) == want, kw
    assert _norm(L, rows=0, x=None, s=None, y=None, ga=None) == da.OK


def _norm_bwd(L, dt=1, sdt=0, rows=12, D=256, x=AT[0], s=AT[1], dy=AT[2], ds=AT[3], gate=AT[4], G=3, scale=1.0, post=1, gp=AT[5], ga=AT[6],
              dx=AT[7], dr=AT[8], dg=AT[9], dgp=AT[10], dga=AT[11], ws=WS, room=ROOM):
    return L.diffattn_residual_norm_backward(dt, sdt, rows, D, x, s, dy, ds, gate, G, F(scale), post, gp, ga, F(1e-5), dx, dr, dg, dgp, dga, ws,
                                             room, None)


def test_norm_backward_refuses(L):
    need = L.diffattn_residual_norm_backward_workspace(12, 256, 3)
    for kw, want in ((dict(dt=0, sdt=1), da.ERR_DTYPE), (dict(D=9000), da.ERR_UNSUPPORTED), (dict(G=7), da.ERR_SHAPE),
                     (dict(dy=None, ds=None, ga=None, dga=None), da.ERR_NULL), (dict(dy=None), da.ERR_SHAPE), (dict(gate=None), da.ERR_SHAPE),
                     (dict(post=0), da.ERR_SHAPE), (dict(post=0, gp=None), da.ERR_SHAPE), (dict(s=None), da.ERR_NULL), (dict(x=None), da.ERR_NULL),
                     (dict(ws=None), da.ERR_NULL), (dict(room=need - 1), da.ERR_SHAPE), (dict(ws=_off(WS, 64)), da.ERR_ALIGN),
                     (dict(dx=_off(AT[7], 8)), da.ERR_ALIGN), (dict(dx=AT[2]), da.ERR_SHAPE), (dict(dr=AT[1]), da.ERR_SHAPE),
                     (dict(dg=AT[4]), da.ERR_SHAPE), (dict(dga=AT[10]), da.ERR_SHAPE), (dict(dr=_off(AT[3], 1024)), da.ERR_SHAPE),
                     (dict(dx=_off(WS, 512)), da.ERR_SHAPE), (dict(scale=float("nan")), da.ERR_SHAPE)):
        assert _norm_bwd(L, **kw) == want, kw
    assert _norm_bwd(L, dx=None, dr=None, dg=None, dgp=None, dga=None) == da.OK


def test_backward_passes_refuse_sizes_whose_indexes_would_overflow(L):
    for kw in (dict(M=0x7ffffff0, N=8, K=8, ldy=8, dx=None, dw=None), dict(M=1, N=0x7ffffff8, K=8, ldy=0x7ffffff8, dx=None, dw=None),
               dict(M=1, N=8, K=0x7ffffff8, ldy=8, lda=0x7ffffff8)):
        assert _linear_bwd(L, **kw) == da.ERR_SHAPE and b"too large" in L.diffattn_last_error(), kw
    for kw in (dict(M=0x7ffffff0, F=8, D=8, ldh=8), dict(M=1, F=0x3ffffff8, D=8, ldh=0x3ffffff8), dict(M=1, F=8, D=0x7ffffff8, ldx=0x7ffffff8, ldh=8)):
        assert _gated_bwd(L, **kw) == da.ERR_SHAPE and b"too large" in L.diffattn_last_error(), kw


def test_workspace_sizes(L):
    for bad in ((0, 8, 8), (8, 0, 8), (-1, 8, 8)):
        assert L.diffattn_linear_backward_workspace(*bad) == 0 and L.diffattn_gated_linear_backward_workspace(*bad) == 0
    assert L.diffattn_residual_norm_backward_workspace(0, 8, 0) == 0 and L.diffattn_residual_norm_backward_workspace(8, 8, -1) == 0
    # room for sums of every CTA, whatever the gate's sharing
    for rows, D in ((1, 1), (12, 33), (300, 256), (1000, 257), (5000, 2048), (77, 8192)):
        least = L.diffattn_residual_norm_backward_workspace(rows, D, 0)
        assert 8 * D <= least <= 8 * D * 152 * 8 + 1024
        for G in (1, rows):
            assert L.diffattn_residual_norm_backward_workspace(rows, D, G) >= least
    assert L.diffattn_linear_backward_workspace(100000, 8192, 64) >= 100000 * 8192 * 2


def test_binding_refuses_host_tensors():
    t = torch.zeros(8, 8, dtype=torch.bfloat16)
    for call in (lambda: da.linear(t, t), lambda: da.linear_backward(t, t, t), lambda: da.gated_linear(t, t),
                 lambda: da.gated_linear_backward(t, t, t, t), lambda: da.residual_norm(t), lambda: da.residual_norm_backward(t, t, t)):
        with pytest.raises(ValueError):
            call()
