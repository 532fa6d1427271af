"""The oracle of the block's operators: its gradients against central differences, its values against plain loops."""

import math

import numpy as np
import pytest

from oracle import block

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def _differences(f, x, dout, h=1e-6):
    """Gradient of sum(dout f(x)) by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + h
        up = float((dout * f()).sum())
        x[i] = keep - h
        g[i] = (up - float((dout * f()).sum())) / (2 * h)
        x[i] = keep
    return g


def _close(a, b):
    assert np.allclose(a, b, rtol=2e-6, atol=2e-7), float(np.max(np.abs(a - b)))


def test_activations_against_their_integrals():
    for z in (-9.0, -3.0, -0.7, 0.0, 0.3, 2.0, 8.0):
        phi = 0.5 * math.erfc(-z / math.sqrt(2))
        assert block.activation(z, "gelu")[0] == pytest.approx(z * phi, rel=1e-9, abs=1e-14)
        assert block.activation(z, "silu")[0] == pytest.approx(z / (1 + math.exp(-z)), rel=1e-12)
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        assert block.activation(z, "gelu_tanh")[0] == pytest.approx(z / (1 + math.exp(-2 * u)), rel=1e-7, abs=1e-14)
    assert block.activation(0.0, "relu") == (0.0, 0.0)


@pytest.mark.parametrize("act", ACTS)
def test_linear_gradients(act):
    r = np.random.default_rng(1)
    a, w, b, dy = r.normal(size=(5, 4)), r.normal(size=(3, 4)), r.normal(size=3), r.normal(size=(5, 3))
    z = block.linear(a, w, b, act)[1]
    da, dw, db, _ = block.linear_backward(a, w, dy, z, act)
    for x, got in ((a, da), (w, dw), (b, db)):
        _close(got, _differences(lambda: block.linear(a, w, b, act)[0], x, dy))


@pytest.mark.parametrize("act", ACTS)
def test_gated_gradients(act):
    r = np.random.default_rng(2)
    x, w, dh = r.normal(size=(4, 3)), r.normal(size=(10, 3)), r.normal(size=(4, 5))
    gu = block.gated_linear(x, w, act)[1]
    dx, dw, _ = block.gated_linear_backward(x, w, gu, dh, act)
    for t, got in ((x, dx), (w, dw)):
        _close(got, _differences(lambda: block.gated_linear(x, w, act)[0], t, dh))


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("G", [0, 1, 2, 6])
def test_norm_gradients(post, G):
    r = np.random.default_rng(3)
    rows, D = 6, 5
    x, res, gp, ga = r.normal(size=(rows, D)), r.normal(size=(rows, D)), r.normal(size=D), r.normal(size=D)
    gate = r.normal(size=(G, D)) if G else None
    dy, ds = r.normal(size=(rows, D)), r.normal(size=(rows, D))
    a = dict(gate=gate, scale=0.6, post=post, gamma_post=gp if post else None, gamma=ga)
    got = block.residual_norm_backward(x, block.residual_norm(x, res, **a)[1], dy, ds, **a)

    def both():
        y, s = block.residual_norm(x, res, **a)
        return np.concatenate([y, s])
    dout = np.concatenate([dy, ds])
    names = [("dx", x), ("dresidual", res), ("dgamma", ga)] + ([("dgamma_post", gp)] if post else []) + (
        [("dgate", gate)] if G else [])
    for name, t in names:
        _close(got[name], _differences(both, t, dout))


def test_norm_by_loops():
    r = np.random.default_rng(4)
    x, res, gate = r.normal(size=(4, 3)), r.normal(size=(4, 3)), r.normal(size=(2, 3))
    y, s = block.residual_norm(x, res, gate=gate, scale=0.5, post=True, eps=1e-3)
    for i in range(4):
        rx = math.sqrt(sum(v * v for v in x[i]) / 3 + 1e-3)
        t = [res[i, j] + 0.5 * gate[i // 2, j] * x[i, j] / rx for j in range(3)]
        rs = math.sqrt(sum(v * v for v in t) / 3 + 1e-3)
        for j in range(3):
            assert s[i, j] == pytest.approx(t[j], rel=1e-12)
            assert y[i, j] == pytest.approx(t[j] / rs, rel=1e-12)
