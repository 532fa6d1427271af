"""Workspaces of the block's backward passes hold what a kernel writes there and nothing else (host only: every call below
is refused for a later fault, so that nothing is launched)."""

import pytest

from differential_attention_03_gb300 import binding as da
from .test_block_refusals import AT, WS, _linear_bwd, _norm_bwd, _off
from .test_block_refusals import L  # noqa: F401  (the fixture)

ACT = {"none": 0, "silu": 4}


def _overlaps(L, status):
    return status == da.ERR_SHAPE and b"overlap" in L.diffattn_last_error()


@pytest.mark.parametrize("M,N,K", [(8192, 8192, 64), (65, 8, 8), (1000, 1304, 1000), (64, 512, 64), (1, 8, 8)])
def test_sizes(L, M, N, K):  # noqa: F811
    f = L.diffattn_linear_backward_workspace_for
    every = L.diffattn_linear_backward_workspace(M, N, K)
    dz = -(-M * N * 2 // 256) * 256
    assert f(M, N, K, 0, 0) == 0
    assert f(M, N, K, 4, 0) == dz
    sums = f(M, N, K, 0, 1)  # partial column sums, of 32 rows or more each; up to 64 rows go straight to the gradient
    assert sums == 0 if M <= 64 else 4 * N <= sums <= 4 * N * -(-M // 32) + 256
    assert f(M, N, K, 4, 1) == dz + sums == every
    assert f(M, N, K, 9, 1) == f(0, N, K, 0, 1) == 0
    assert da.linear_backward_workspace_bytes(M, N, K) == every
    assert da.linear_backward_workspace_bytes(M, N, K, "none", False) == 0
    assert da.linear_backward_workspace_bytes(M, N, K, "none", True) == sums
    assert da.linear_backward_workspace_bytes(M, N, K, "gelu", False) == dz


def test_linear_backward_takes_what_it_needs(L):  # noqa: F811
    f = L.diffattn_linear_backward_workspace_for
    late = dict(dx=AT[2])  # (da over dy: found behind the workspace)
    # up to 64 rows without an activation: none at all
    assert _overlaps(L, _linear_bwd(L, M=64, act=0, pre=None, ws=None, room=0, **late))
    for M, act, db in ((100, 0, AT[6]), (100, 4, AT[6]), (100, 4, None), (64, 4, AT[6])):
        need = f(M, 256, 128, act, 1 if db else 0)
        assert need > 0
        assert _overlaps(L, _linear_bwd(L, M=M, act=act, db=db, room=need, **late))
        assert _linear_bwd(L, M=M, act=act, db=db, room=need - 1, **late) == da.ERR_SHAPE and b"workspace" in L.diffattn_last_error()
        assert _linear_bwd(L, M=M, act=act, db=db, ws=None, **late) == da.ERR_NULL
        # no output may lie in what is used of it, and what lies behind is free
        assert _overlaps(L, _linear_bwd(L, M=M, act=act, db=db, dx=_off(WS, need - 256)))


def test_norm_backward_with_a_gate_a_row_needs_no_partial_gates(L):  # noqa: F811
    f = L.diffattn_residual_norm_backward_workspace
    for rows, D in ((700, 128), (1500, 512), (5000, 2048), (37, 33)):
        assert f(rows, D, rows) == f(rows, D, 0)
        assert f(rows, D, 1) >= f(rows, D, 0)
    need = f(12, 256, 12)
    late = dict(G=12, dx=AT[2])
    assert _overlaps(L, _norm_bwd(L, room=need, **late))
    assert _norm_bwd(L, room=need - 1, **late) == da.ERR_SHAPE and b"workspace" in L.diffattn_last_error()


def test_norm_backward_spreads_the_most_rows_over_the_card(L):  # noqa: F811
    """Sums of as many CTAs for 2^31 - 1 rows as for a million: the count of rows does not overflow on the way."""
    f = L.diffattn_residual_norm_backward_workspace
    for D in (1, 8, 33, 256, 512, 2048):
        assert f(0x7fffffff, D, 0) == f(1 << 20, D, 0)


def test_sizes_near_2_to_the_31(L):  # noqa: F811
    """Column sums of the most rows: as many chunks as any other long tensor's.  Plans of sizes past 31 bits are refused."""
    f = L.diffattn_linear_backward_workspace_for
    assert f(0x7fffffff, 264, 8, 0, 1) == f(1 << 20, 264, 8, 0, 1)
    assert f(100, 0x7ffffff8, 8, 0, 1) == 0  # (so many columns that one chunk fills the card: straight to the gradient)
    for sizes in ((0x7fffffff, 8, 8), (8, 0x7ffffff8, 8), (8, 8, 0x7ffffff8)):
        with pytest.raises(ValueError):
            da.debug_product_plan("linear", *sizes)
    assert da.debug_product_plan("linear", 0x7fff0000, 8, 8)["kernel"] in ("few", "tiles")
