"""The per-head norm and rotary positions in 64 bits, one row at a time in the formulas' own
terms: the reference of the kernels' tests."""
from __future__ import annotations

import numpy as np


def pair_columns(rot: int, interleaved: bool):
    """Columns (e, f) of each rotation."""
    p = np.arange(rot // 2)
    return (2 * p, 2 * p + 1) if interleaved else (p, p + rot // 2)


def angles(positions, inv_freq, pair_axis):
    """(rows, rot/2) angles of rows with positions (axes, rows)."""
    axis = np.zeros(len(inv_freq), int) if pair_axis is None else np.asarray(pair_axis, int)
    return np.asarray(positions, np.float64)[axis].T * np.asarray(inv_freq, np.float64)


def turn(x, ang, interleaved, sign=1.0):
    """Rotates the rows' pairs by sign * ang; x (rows, heads, d), ang (rows, rot/2)."""
    y = x.copy()
    e, f = pair_columns(2 * ang.shape[1], interleaved)
    c, s = np.cos(ang)[:, None, :], sign * np.sin(ang)[:, None, :]
    y[..., e] = x[..., e] * c - x[..., f] * s
    y[..., f] = x[..., f] * c + x[..., e] * s
    return y


def forward(x, gain, ang, interleaved, norm, eps):
    """x (rows, heads, d) -> y; gain (d,) or None."""
    u = x
    if norm:
        u = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if gain is not None:
            u = u * gain
    return turn(u, ang, interleaved)


def backward(dy, x, gain, ang, interleaved, norm, eps):
    """(dx, dgain, sum |terms of dgain|) from dy, x (rows, heads, d)."""
    g = turn(dy, ang, interleaved, -1.0)
    if not norm:
        return g, None, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    t = g if gain is None else g * gain
    dx = r * (t - xh * (t * xh).mean(-1, keepdims=True))
    return dx, (g * xh).sum((0, 1)), np.abs(g * xh).sum((0, 1))
