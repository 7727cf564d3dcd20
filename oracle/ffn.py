"""Gated feed-forward block in float64 (test infrastructure only): s = act(g) * u of [g | u] = x W_up, y = s W_down,
and its backward on the kept rows.  Beside each result stands what may be lost of it: the sum of the magnitudes that
its rounded factors meet, by which a test counts roundings."""
from __future__ import annotations

import numpy as np

C1, C3 = np.sqrt(2.0 / np.pi), 0.044715


def act(g, kind):
    """a(g) and a'(g)."""
    g = np.asarray(g, np.float64)
    with np.errstate(over="ignore"):
        if kind == "silu":
            p = 1.0 / (1.0 + np.exp(-g))
            return g * p, p + g * p * (1.0 - p)
        t = np.tanh(C1 * (g + C3 * g ** 3))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * C1 * (1.0 + 3.0 * C3 * g * g)


def forward(x, w_up, w_down, kind):
    x, w_up, w_down = (np.asarray(v, np.float64) for v in (x, w_up, w_down))
    up = x @ w_up
    g, u = np.split(up, 2, axis=1)
    s = act(g, kind)[0] * u
    return dict(up=up, s=s, y=s @ w_down)


def backward(x, up, dy, w_up, w_down, kind, keep=None):
    """keep: boolean [M] (None: all).  Rows of filtered tokens count for nothing and get a dx of 0."""
    x, up, dy, w_up, w_down = (np.asarray(v, np.float64) for v in (x, up, dy, w_up, w_down))
    if keep is not None:
        m = np.asarray(keep, bool)[:, None]
        x, up, dy = np.where(m, x, 0.0), np.where(m, up, 0.0), np.where(m, dy, 0.0)
    g, u = np.split(up, 2, axis=1)
    a, da = act(g, kind)
    ds = dy @ w_down.T
    dup = np.concatenate((ds * u * da, ds * a), axis=1)
    return dict(dup=dup, s=a * u, dx=dup @ w_up.T, dw_up=x.T @ dup, dw_down=(a * u).T @ dy)
