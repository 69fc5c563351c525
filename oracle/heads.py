"""Heads between a block's projections in 64 bits: norm and rotation with their gradients, the 8-bit form of a cache, attention over
pages. Plain numpy from the definitions; shares no code with the library."""
from __future__ import annotations

import math

import numpy as np


def turns(rot, base, kind="plain", factor=1.0, original=0.0, low=1.0, high=4.0):
    """Turns per position of each pair, as real numbers."""
    if kind == "base":
        base = base * factor ** (rot / (rot - 2))
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot) / (2 * math.pi)
        if kind == "linear":
            f /= factor
        elif kind in ("parts", "by_index"):
            if kind == "parts":
                s = (original * f - low) / (high - low)
            else:
                at = [rot / 2 * math.log(original / (2 * math.pi * r)) / math.log(base) for r in (low, high)]
                s = (at[0] - i) / (at[0] - at[1])
            s = min(max(s, 0.0), 1.0)
            f = s * f + (1 - s) * f / factor
        out.append(f)
    return np.array(out)


def angle(pos, fractions):
    """Radians [tokens, pairs]: whole numbers modulo a turn of 2^64, exactly."""
    a = [[(int(p) * int(f)) % (1 << 64) for f in fractions] for p in pos]
    return np.array(a, dtype=np.float64).reshape(len(pos), len(fractions)) * (2 * math.pi / 2.0 ** 64)


def _members(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(x, theta, interleaved, amplitude=1.0):
    """x [T, H, D] with its pairs turned by theta [T, R / 2]."""
    y = x.copy()
    a, b = _members(2 * theta.shape[1], interleaved)
    c, s = amplitude * np.cos(theta)[:, None], amplitude * np.sin(theta)[:, None]
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return y


def norm(x, w, eps):
    y = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    return y if w is None else y * w


def forward(x, w, eps, theta, interleaved, amplitude=1.0, normed=True):
    return rotate(norm(x, w, eps) if normed else x, theta, interleaved, amplitude)


def backward(dy, x, w, eps, theta, interleaved, amplitude=1.0, normed=True):
    """dx and dw (None without a norm)."""
    d = rotate(dy, -theta, interleaved, amplitude)
    if not normed:
        return d, None
    r = 1 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    z = x * r
    dz = d if w is None else d * w
    return r * (dz - z * (dz * z).mean(axis=-1, keepdims=True)), (d * z).sum(axis=(0, 1))


def e4m3_values():
    """The value of each code."""
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v[c] = (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)) * (-1 if c & 128 else 1)
        if c & 127 == 127:
            v[c] = np.nan
    return v


def mx_exponents(x):
    """e of each group of 32 along the last axis (NaN groups: 128, the byte 0xFF)."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    a = np.abs(g)
    a = np.where(np.isinf(a), 255 * 2.0 ** 120, a).max(axis=-1)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.ceil(np.log2(a / 448))
        e = np.where(448 * np.exp2(e) < a, e + 1, np.where(448 * np.exp2(e - 1) >= a, e - 1, e))
    e = np.where(a == 0, 0, np.maximum(e, -127))
    return np.where(np.isnan(a), 128, e).astype(int)


def mx_decode(codes, units):
    """The values of uint8 codes [..., D] with scale bytes [..., D / 32]."""
    f = np.where(units == 255, np.nan, np.exp2(units.astype(np.float64) - 127))
    return e4m3_values()[codes] * np.repeat(f, 32, axis=-1)


def places(q_start, kv_len, tokens):
    """(sequence, position) of each row; (-1, -1) for rows of nobody."""
    out = [(-1, -1)] * tokens
    for s in range(len(kv_len)):
        lo, hi = max(0, int(q_start[s])), min(tokens, int(q_start[s + 1]))
        for t in range(lo, hi):
            out[t] = (s, max(0, int(kv_len[s])) - (hi - lo) + t - lo)
    return out


def attention(q, k, v, q_start, kv_len, table, scale, window=0):
    """q [T, Hq, D]; k and v [pages, Hk, page, D], all in 64 bits. Returns out, lse, and the sums that error bounds are made of: sum of
    w |v| / sum of w, and the largest scale sum |q k| of each row. Rows of nobody are NaN."""
    T, Hq, D = q.shape
    pages, Hk, P, _ = k.shape
    G = Hq // Hk
    out, lse = np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    mag, big = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for t, (s, p) in enumerate(places(q_start, kv_len, T)):
        if s < 0:
            continue
        end = min(p + 1, table.shape[1] * P, max(0, int(kv_len[s])))
        j = np.arange(max(0, p + 1 - window) if window else 0, max(end, 0))
        out[t], lse[t] = 0.0, -np.inf
        if len(j) == 0:
            continue
        page = table[s, j // P]
        good = (page >= 0) & (page < pages)
        at = np.where(good, page, 0)
        for h in range(Hq):
            kk = np.where(good[:, None], k[at, h // G, j % P], 0.0)
            vv = np.where(good[:, None], v[at, h // G, j % P], 0.0)
            with np.errstate(invalid="ignore", over="ignore"):
                w = scale * (kk @ q[t, h])
                big[t, h] = abs(scale) * np.max(np.abs(kk) @ np.abs(q[t, h]))
                top = np.max(w)
                e = np.exp(w - (top if np.isfinite(top) else 0.0))
                out[t, h], mag[t, h] = (e @ vv) / e.sum(), (e @ np.abs(vv)) / e.sum()
                lse[t, h] = top + np.log(e.sum())
    return out, lse, mag, big
