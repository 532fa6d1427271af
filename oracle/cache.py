"""Positions, cache formats, draft trees and accepted paths in fp64 on the CPU (loops, no cleverness)."""

import math

import numpy as np

from .diffattn_oracle import _f64, e4m3_decode, head_rmsnorm


def rope_frequencies(rot, base=10000.0, scaling="none", factor=1.0, original=0, beta_fast=32.0, beta_slow=1.0):
    """(theta [rot / 2], factor on the rotated channels)."""
    if scaling == "ntk":
        base *= factor ** (rot / (rot - 2))
    th = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        th = [t / factor for t in th]
    if scaling == "yarn":
        def pair(beta):
            return rot * math.log(original / (2 * math.pi * beta)) / (2 * math.log(base))
        low, high = max(0, math.floor(pair(beta_fast))), min(rot - 1, math.ceil(pair(beta_slow)))
        for i in range(rot // 2):
            w = min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
            th[i] = th[i] * (1 - w) + th[i] / factor * w
        return np.array(th), 0.1 * math.log(factor) + 1.0
    return np.array(th), 1.0


def rope(x, pos, th, mult=1.0, interleaved=False, inverse=False):
    """x [B, n, heads, d], pos [B, n]."""
    x = _f64(x)
    y = x.copy()
    half = len(th)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ang = np.asarray(pos, np.float64)[..., None] * th[i] * (-1.0 if inverse else 1.0)
        c, s = mult * np.cos(ang), mult * np.sin(ang)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def e4m3_round(x):
    """Nearest finite e4m3 value, ties to the even code, saturating at 448 (x any shape, fp64)."""
    table = np.array([e4m3_decode(np.array([c], np.uint8))[0] for c in range(127)])  # ascending, code 127 is NaN
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(table, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - table[lo], table[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.copysign(table[pick], x)


def quantise_rows(x):
    """(values on the e4m3 grid, scale) of each row (last axis)."""
    x = _f64(x)
    scale = np.abs(x).max(-1) / 448.0
    safe = np.where(scale > 0, scale, 1.0)
    return e4m3_round(x / safe[..., None]), scale


def sees(L, nt, T, n, mask):
    """[T, n] truth values: what drafted token t sees; mask: T words or None for a chain."""
    out = np.zeros((T, n), bool)
    for t in range(min(T, nt)):
        out[t, :L] = True
        for u in range(nt):
            if L + u < n and (u <= t if mask is None else (int(mask[t]) >> u) & 1):
                out[t, L + u] = True
    return out


def _map(q, k, v, seen, scale):
    """(O [T, dv], sum_j p |v|, largest weight) of one map."""
    T = q.shape[0]
    o = np.zeros((T, v.shape[1]))
    a = np.zeros_like(o)
    w = np.zeros(T)
    for t in range(T):
        j = np.nonzero(seen[t])[0]
        if len(j) == 0:
            continue
        s = k[j] @ q[t] * scale
        p = np.exp(s - s.max())
        p /= p.sum()
        o[t], a[t] = p @ v[j], p @ np.abs(v[j])
        w[t] = (p * np.abs(v[j]).max(-1)).max()
    return o, a, w


def tree_v1(q1, q2, k1, k2, v, lens, ntok, mask, lam, lam_init, gamma, eps):
    """q [B, T, H, d], caches [B, n, H, .] as the values they stand for.  Returns (out, bound's parts):
    out [B, T, H, 2d], and per element sum_r c_r sum_j p |v| and per row sum_r c_r max_j p |v| with
    c = (1, |lam|), before the norm, and the norm's factor per element."""
    q1, q2, k1, k2, v = (_f64(x) for x in (q1, q2, k1, k2, v))
    B, T, H, d = q1.shape
    n = k1.shape[1]
    out = np.zeros((B, T, H, 2 * d))
    spread, top, pre, gain = np.zeros_like(out), np.zeros((B, T, H)), np.zeros_like(out), np.zeros_like(out)
    for b in range(B):
        seen = sees(lens[b], ntok[b], T, n, None if mask is None else mask[b])
        for h in range(H):
            o1, a1, w1 = _map(q1[b, :, h], k1[b, :, h], v[b, :, h], seen, 1 / math.sqrt(d))
            o2, a2, w2 = _map(q2[b, :, h], k2[b, :, h], v[b, :, h], seen, 1 / math.sqrt(d))
            o = o1 - lam * o2
            out[b, :, h] = head_rmsnorm(o, gamma, eps, lam_init)
            pre[b, :, h] = o
            spread[b, :, h] = a1 + abs(lam) * a2
            top[b, :, h] = w1 + abs(lam) * w2
            gain[b, :, h] = (1 - lam_init) * np.abs(_f64(gamma)) / np.sqrt((o * o).mean(-1, keepdims=True) + eps)
    return out, pre, spread, top, gain


def tree_v2(q, k, v, logits, lens, ntok, mask, scale=None):
    """q [B, T, Hq, d], caches [B, n, Hkv, d], logits [B, T, Hq / 2].  Returns (out, spread, top)."""
    q, k, v, logits = (_f64(x) for x in (q, k, v, logits))
    B, T, Hq, d = q.shape
    n, Hkv = k.shape[1], k.shape[2]
    scale = 1 / math.sqrt(d) if scale is None else scale
    out = np.zeros((B, T, Hq // 2, d))
    spread, top = np.zeros_like(out), np.zeros((B, T, Hq // 2))
    for b in range(B):
        seen = sees(lens[b], ntok[b], T, n, None if mask is None else mask[b])
        for g in range(Hq // 2):
            h = 2 * g // (Hq // Hkv)
            o1, a1, w1 = _map(q[b, :, 2 * g], k[b, :, h], v[b, :, h], seen, scale)
            o2, a2, w2 = _map(q[b, :, 2 * g + 1], k[b, :, h], v[b, :, h], seen, scale)
            c = 1 / (1 + np.exp(-logits[b, :, g]))
            out[b, :, g] = o1 - c[:, None] * o2
            spread[b, :, g] = a1 + c[:, None] * a2
            top[b, :, g] = w1 + c * w2
    return out, spread, top
