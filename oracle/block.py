"""What stands around the attention layer in a block, in fp64 on the CPU: products, activations, norms, gradients."""

import numpy as np
from scipy.special import erf

from .diffattn_oracle import _f64

_C0, _C1 = np.sqrt(2 / np.pi), 0.044715


def activation(z, act):
    """(act(z), act'(z))."""
    z = np.asarray(z, np.float64)
    if act == "none":
        return z, np.ones_like(z)
    if act == "relu":
        return np.maximum(z, 0.0), (z > 0).astype(np.float64)
    if act == "gelu":
        phi = 0.5 * (1 + erf(z / np.sqrt(2)))
        return z * phi, phi + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    if act == "gelu_tanh":
        t = np.tanh(_C0 * (z + _C1 * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * _C0 * (1 + 3 * _C1 * z * z)
    w = 0.5 * (1 + np.tanh(z / 2))
    return z * w, w * (1 + z * (1 - w))


def linear(a, w, bias=None, act="none", residual=None):
    """(out, z): z = a w^T + bias, out = residual + act(z)."""
    z = _f64(a) @ _f64(w).T
    if bias is not None:
        z = z + _f64(bias)
    out = activation(z, act)[0]
    return (out if residual is None else out + _f64(residual)), z


def linear_backward(a, w, dy, z=None, act="none"):
    """(da, dw, dbias, dz)."""
    dz = _f64(dy)
    if act != "none":
        dz = dz * activation(_f64(z), act)[1]
    return dz @ _f64(w), dz.T @ _f64(a), dz.sum(0), dz


def gated_linear(x, w_gu, act="silu"):
    """(h, gu): gu = x w_gu^T = [g | u], h = act(g) u."""
    gu = _f64(x) @ _f64(w_gu).T
    F = gu.shape[1] // 2
    return activation(gu[:, :F], act)[0] * gu[:, F:], gu


def gated_linear_backward(x, w_gu, gu, dh, act="silu"):
    """(dx, dw, dgu)."""
    gu, dh = _f64(gu), _f64(dh)
    F = gu.shape[1] // 2
    value, slope = activation(gu[:, :F], act)
    dgu = np.concatenate([dh * gu[:, F:] * slope, dh * value], 1)
    return dgu @ _f64(w_gu), dgu.T @ _f64(x), dgu


def _rms(x, eps):
    return 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def _rows_of(gate, rows):
    """A gate of G rows as one row for each of `rows`."""
    gate = _f64(gate)
    gate = gate.reshape(-1, gate.shape[-1])
    return np.repeat(gate, rows // gate.shape[0], 0)


def residual_norm(x, residual=None, gate=None, scale=1.0, post=False, gamma_post=None, gamma=None, eps=1e-5):
    """(y, s) of rows x [rows, D]; gate [G, D], G dividing the rows."""
    x = _f64(x)
    p = x
    if post:
        p = x * _rms(x, eps) * (1.0 if gamma_post is None else _f64(gamma_post))
    if gate is not None:
        p = p * _rows_of(gate, x.shape[0])
    s = scale * p + (0.0 if residual is None else _f64(residual))
    return s * _rms(s, eps) * (1.0 if gamma is None else _f64(gamma)), s


def residual_norm_backward(x, s, dy=None, ds=None, gate=None, scale=1.0, post=False, gamma_post=None, gamma=None,
                           eps=1e-5):
    """dict of dx, dresidual, dgate [G, D], dgamma_post, dgamma (those that apply)."""
    x, s = _f64(x), _f64(s)
    rows, D = x.shape
    t = np.zeros_like(x) if ds is None else _f64(ds).copy()
    r = {}
    if dy is not None:
        dy, rs = _f64(dy), _rms(s, eps)
        n = s * rs
        dn = dy * (1.0 if gamma is None else _f64(gamma))
        t += rs * (dn - n * (dn * n).mean(-1, keepdims=True))
        r["dgamma"] = (dy * n).sum(0)
    r["dresidual"] = t
    g = 1.0 if gate is None else _rows_of(gate, rows)
    dp = scale * t * g
    if post:
        gp = 1.0 if gamma_post is None else _f64(gamma_post)
        rx = _rms(x, eps)
        xh = x * rx
        p, dn = xh * gp, dp * gp
        r["dgamma_post"] = (dp * xh).sum(0)
        r["dx"] = rx * (dn - xh * (dn * xh).mean(-1, keepdims=True))
    else:
        p, r["dx"] = x, dp
    if gate is not None:
        G = _f64(gate).reshape(-1, D).shape[0]
        r["dgate"] = (scale * t * p).reshape(G, rows // G, D).sum(1)
    return r
