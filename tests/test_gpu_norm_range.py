"""Norms of rows whose squares leave fp32's range, beside rows that stay in it, in every layout of a row.

Elements of 1e19: their squares' sum is above 3.4e38, so such a row is summed again scaled.  Its statistics are then as
accurate as any other row's, and the bounds are those of test_gpu_block.py.  Gradients of such rows are of the size of
dy / 1e19, so dy is of that size there, and what comes out is around one.
"""

import pytest
import torch

from differential_attention_03_gb300 import binding as da
from .test_gpu_block import TYPES, _check_norm, _check_norm_backward

pytestmark = pytest.mark.gpu

F32 = torch.float32
ROWS, BIG = 37, 1e19
# sub-warp, warp (odd, even), ring of one vector, CTA (odd, even), ring of two or pairs, CTA above 4096 (odd, even), ring above
WIDTHS = [64, 33, 250, 504, 1001, 1002, 2048, 4099, 5002, 8192]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from differential_attention_03_gb300 import build
    build.build()
    torch.cuda.init()


def _inputs(D, types, gates):
    g = torch.Generator(device="cuda").manual_seed(D + gates)
    dt, sdt = TYPES[types]

    def rnd(*shape, big=(), dtype=F32):
        t = torch.randn(shape, generator=g, device="cuda")
        for r in big:
            t[r::7] *= BIG
        return t.to(dtype)
    gate = None if gates == 0 else 1 + 0.3 * rnd(gates, D)
    return rnd, dt, sdt, gate, 1 + 0.1 * rnd(D), 1 + 0.1 * rnd(D)


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("gates", [0, 1, ROWS])
@pytest.mark.parametrize("post", [False, True])
def test_rows_of_large_elements(D, types, gates, post):
    rnd, dt, sdt, gate, gp, ga = _inputs(D, types, gates)
    x, res = rnd(ROWS, D, big=(2, 5), dtype=dt), rnd(ROWS, D, big=(2, 4), dtype=sdt)
    gp = gp if post else None
    y, s = da.residual_norm(x, res, gate=gate, scale=0.5, gamma_post=gp, gamma=ga)
    assert torch.isfinite(y).all() and torch.isfinite(s).all()
    _check_norm(x, res, gate, gp, ga, 0.5, y, s)
    da.device_status()


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("gates", [0, 1, ROWS])
@pytest.mark.parametrize("post", [False, True])
def test_gradients_of_rows_of_large_elements(D, types, gates, post):
    """Rows 2, 9, ..: s and dy large; 5, 12, ..: s, x and dy; with post 3, 10, ..: x and dy, so that dy's size reaches dx."""
    rnd, dt, sdt, gate, gp, ga = _inputs(D, types, gates)
    x = rnd(ROWS, D, big=(3, 5) if post else (), dtype=dt)
    s = rnd(ROWS, D, big=(2, 5), dtype=sdt)
    dy = rnd(ROWS, D, big=(2, 3, 5) if post else (2, 5), dtype=dt)
    ds = rnd(ROWS, D, dtype=sdt)
    gp = gp if post else None
    got = da.residual_norm_backward(x, s, dy, ds, gate=gate, scale=0.5, gamma_post=gp, gamma=ga)
    assert all(torch.isfinite(t).all() for t in got.values())
    _check_norm_backward(x, s, dy, ds, gate, gp, ga, 0.5, got)
    # the rows' own gradients are not lost beside zeros
    assert float(got["dx"][2::7].abs().float().mean()) > 0.05 and float(got["dresidual"][5::7].abs().float().mean()) > 0.05
    da.device_status()


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("gates", [0, 1, ROWS])
def test_elements_near_the_types_largest(D, types, gates):
    """Elements of 2.5e38 are normed before gamma and the gate, above one here, multiply them."""
    g = torch.Generator(device="cuda").manual_seed(D)
    dt, sdt = TYPES[types]
    x = (2.5e38 * (1 - 0.2 * torch.rand(ROWS, D, generator=g, device="cuda"))).to(dt)
    x[::3] = torch.randn(x[::3].shape, generator=g, device="cuda").to(dt)
    gate = None if gates == 0 else 2 + torch.rand(gates, D, generator=g, device="cuda")
    gp, ga = (3 + torch.rand(D, generator=g, device="cuda") for _ in range(2))
    res = torch.randn(ROWS, D, generator=g, device="cuda").to(sdt)
    y, s = da.residual_norm(x, res, gate=gate, scale=0.5, gamma_post=gp, gamma=ga)
    assert torch.isfinite(y).all() and torch.isfinite(s).all()
    _check_norm(x, res, gate, gp, ga, 0.5, y, s)
    got = da.residual_norm_backward(x, s, res.to(dt), res, gate=gate, scale=0.5, gamma_post=gp, gamma=ga)
    assert all(torch.isfinite(t).all() for t in got.values())
    _check_norm_backward(x, s, res.to(dt), res, gate, gp, ga, 0.5, got)
    da.device_status()
