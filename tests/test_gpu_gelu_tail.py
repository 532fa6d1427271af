"""gelu in its tail: small values keep their relative accuracy, in both product kernels and in the gradients.

Phi(-|z|) = e t P(t), e = exp(-z^2 / 2): three roundings of the exponent (the square, log2 e / 2, their product), 2^-24 each,
cost 3 * 2^-24 z^2 / 2 of e; the exponential 2^-22; the polynomial 3e-7 and the four products and roundings behind it 2^-22
more: in fp32 2^-20 + 1.5 z^2 2^-24 of the value.  In bf16 the polynomial is within 5e-6 (2^-17) and the result's rounding 2^-8.
"""

import math

import numpy as np
import pytest
import torch
from scipy.special import erfc

from differential_attention_03_gb300 import binding as da

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from differential_attention_03_gb300 import build
    build.build()
    torch.cuda.init()


def _values():
    """bf16 values, both signs, to where the tail leaves fp32; a multiple of 8 of them."""
    z = torch.cat([torch.linspace(0.0, 4.0, 200), torch.linspace(4.0, 12.9, 152)]).to(BF)
    return torch.cat([z, -z])


def _phi(z):
    return 0.5 * erfc(-z / math.sqrt(2))


def _rows(z, M):
    """Operands whose product is z in each of M rows."""
    w = torch.zeros(z.numel(), 8, dtype=BF)
    w[:, 0] = z
    a = torch.zeros(M, 8, dtype=BF)
    a[:, 0] = 1
    return a.cuda(), w.cuda()


@pytest.mark.parametrize("M", [3, 300, 70000])
def test_gelu_tail(M):
    z = _values()
    Z = z.double().numpy()
    a, w = _rows(z, M)
    if M > 1000:
        assert da.debug_product_plan("linear", M, z.numel(), 8)["kernel"] == "tiles"
    ref = Z * _phi(Z)
    for dtype, bound in ((F32, 2.0 ** -20 + 1.5 * Z * Z * 2.0 ** -24), (BF, 2.0 ** -8 + 2.0 ** -17 + 1.5 * Z * Z * 2.0 ** -24)):
        got = da.linear(a, w, act="gelu", dtype=dtype)
        assert torch.equal(got[0], got[-1])
        err = np.abs(got[M // 2].double().cpu().numpy() - ref)
        assert np.all(err <= bound * np.abs(ref) + 1e-37), (dtype, Z[np.argmax(err / (bound * np.abs(ref) + 1e-37))])
    da.device_status()


@pytest.mark.parametrize("M", [3, 70000])
def test_gated_gelu_tail(M):
    z = _values()
    Z = z.double().numpy()
    a, w = _rows(z, M)
    up = torch.zeros_like(w)
    up[:, 0] = 1
    h = da.gated_linear(a, torch.cat([w, up]), act="gelu")
    ref = Z * _phi(Z)
    assert np.all(np.abs(h[0].double().cpu().numpy() - ref) <= (2.0 ** -8 + 2.0 ** -17 + 1.5 * Z * Z * 2.0 ** -24) * np.abs(ref) + 1e-37)
    da.device_status()


def test_gelu_slope_tail():
    """The slope Phi + z phi in fp32 (as a bias gradient of one row): its two terms cancel in the tail, so it is held to their
    magnitudes."""
    z = _values()
    Z, N = z.double().numpy(), z.numel()
    one = torch.ones(1, N, dtype=BF, device="cuda")
    w = torch.zeros(N, 8, dtype=BF, device="cuda")
    x = torch.zeros(1, 8, dtype=BF, device="cuda")
    got = da.linear_backward(x, w, one, pre=z[None].cuda(), act="gelu", bias=True, da=False, dw=False)["dbias"].double().cpu().numpy()
    phi = np.exp(-Z * Z / 2) / math.sqrt(2 * math.pi)
    size = _phi(Z) + np.abs(Z) * phi
    assert np.all(np.abs(got - (_phi(Z) + Z * phi)) <= (2.0 ** -20 + 1.5 * Z * Z * 2.0 ** -24) * size + 1e-37)
    da.device_status()
