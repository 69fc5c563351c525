"""The norms around a block with its gate and the residual's scale (oracle; test infrastructure):
forward and backward from the formulas, in fp64.

    n = norm_post(o) w_post + b_post;  r' = alpha r + gate n;  h = norm_pre(r') w_pre + b_pre

Pins: tests/test_oracle_norm.py (closed forms; the gradients against central differences).
"""
from __future__ import annotations

import numpy as np

NONE, RMS, LAYER = 0, 1, 2


def stat(x, kind, eps):
    """(mean, 1 / root) per row, [T, 1] each."""
    t = x.shape[0]
    if kind == NONE:
        return np.zeros((t, 1)), np.ones((t, 1))
    mean = x.mean(axis=1, keepdims=True) if kind == LAYER else np.zeros((t, 1))
    with np.errstate(all="ignore"):
        return mean, 1.0 / np.sqrt(((x - mean) ** 2).mean(axis=1, keepdims=True) + eps)


def _affine(z, w, b):
    z = z if w is None else z * w
    return z if b is None else z + b


def gate_rows_of(gate, rows, t):
    return None if gate is None else gate[np.arange(t) // rows]


def forward(r, o=None, gate=None, gate_rows=1, alpha=1.0, post=NONE, pre=RMS, eps=1e-5, w_post=None, b_post=None, w_pre=None, b_pre=None):
    """{"r", "h", "post": (mean, inv), "pre": (mean, inv)}."""
    out = r * alpha
    sp = (np.zeros((len(r), 1)), np.ones((len(r), 1)))
    if o is not None:
        sp = stat(o, post, eps)
        n = _affine((o - sp[0]) * sp[1], w_post, b_post)
        g = gate_rows_of(gate, gate_rows, len(r))
        out = out + (n if g is None else g * n)
    sq = stat(out, pre, eps)
    return {"r": out, "h": _affine((out - sq[0]) * sq[1], w_pre, b_pre), "post": sp, "pre": sq}


def _norm_back(dy, x, st, w, kind):
    if kind == NONE:
        return dy, None, None
    z = (x - st[0]) * st[1]
    dz = dy if w is None else dy * w
    dx = dz - z * (dz * z).mean(axis=1, keepdims=True)
    if kind == LAYER:
        dx = dx - dz.mean(axis=1, keepdims=True)
    return dx * st[1], (dy * z).sum(axis=0), dy.sum(axis=0)


def backward(r, r_out, dh, dr_out, o=None, gate=None, gate_rows=1, alpha=1.0, post=NONE, pre=RMS, st_post=None, st_pre=None,
             w_post=None, b_post=None, w_pre=None, b_pre=None):
    """Every gradient, from the stored stream r_out and the statistics; dh or dr_out may be None."""
    t, d = r_out.shape
    g = np.zeros((t, d)) if dr_out is None else dr_out.copy()
    dw_pre = db_pre = np.zeros(d)
    if dh is not None:
        dx, dw, db = _norm_back(dh, r_out, st_pre, w_pre, pre)
        g = g + dx
        if pre != NONE:
            dw_pre, db_pre = dw, db
    res = {"dr": alpha * g, "dscale": (g * r).sum(), "dw_pre": dw_pre, "db_pre": db_pre, "g": g}
    if o is not None:
        gr = gate_rows_of(gate, gate_rows, t)
        z = (o - st_post[0]) * st_post[1]
        if gr is not None:
            res["dgate"] = np.zeros(gate.shape)
            np.add.at(res["dgate"], np.arange(t) // gate_rows, g * _affine(z, w_post, b_post))
        dn = g if gr is None else g * gr
        res["do"], res["dw_post"], res["db_post"] = _norm_back(dn, o, st_post, w_post, post)
    return res
