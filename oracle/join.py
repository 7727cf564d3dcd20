"""Residual join (norms after and before a block's branch, gate, residual scale) and its backward on the kept
rows, in float64 (test infrastructure only).

  h = alpha lam . x + gate_b . post(y),   a = pre(h)

post and pre are RMSNorm or LayerNorm.  The backward takes the saved rows and row statistics as given, as the
library does: it differentiates v -> w (v - m) r + b at those values.
"""
from __future__ import annotations

import numpy as np


def stats(v, ln, eps):
    m = v.mean(axis=1) if ln else np.zeros(v.shape[0])
    r = 1.0 / np.sqrt(np.mean((v - m[:, None]) ** 2, axis=1) + eps)
    return m, r


def norm(v, m, r, w, b):
    return (v - m[:, None]) * r[:, None] * w + (0.0 if b is None else b)


def gate_rows(gate, B, T, D):
    """The gate of each token: gate None (1), [1, D] or [B, D]."""
    if gate is None:
        return np.ones((B * T, D))
    return np.repeat(np.broadcast_to(gate, (B, D)), T, axis=0)


def join_forward(x, y, p, B, T, alpha, ln, eps, store=lambda v: v):
    """p: dict post_w, post_b, gate, res_w, pre_w, pre_b (None where absent; no post norm without post_w, no a
    without pre_w).  store rounds h.  Returns dict h, a, mean_y, rstd_y, mean_h, rstd_h."""
    out = {}
    D = x.shape[1]
    if y is None:
        h = x
    else:
        branch = y
        if p["post_w"] is not None:
            out["mean_y"], out["rstd_y"] = stats(y, ln, eps)
            branch = norm(y, out["mean_y"], out["rstd_y"], p["post_w"], p["post_b"])
        lam = 1.0 if p["res_w"] is None else p["res_w"]
        h = store(alpha * lam * x + gate_rows(p["gate"], B, T, D) * branch)
        out["h"] = h
    if p["pre_w"] is not None:
        out["mean_h"], out["rstd_h"] = stats(h, ln, eps)
        out["a"] = norm(h, out["mean_h"], out["rstd_h"], p["pre_w"], p["pre_b"])
    return out


def _norm_input_grad(t, hat, r, ln):
    """t = gradient of the normalised row hat -> gradient of the row; and the sum of the magnitudes of its terms."""
    k = np.mean(t * hat, axis=1, keepdims=True)
    g = t - hat * k
    mag = np.abs(t) + np.abs(hat) * np.mean(np.abs(t * hat), axis=1, keepdims=True)
    if ln:
        g = g - t.mean(axis=1, keepdims=True)
        mag = mag + np.mean(np.abs(t), axis=1, keepdims=True)
    return g * r[:, None], mag * r[:, None]


def join_backward(x, y, h, st, da, dh, p, B, T, keep, alpha, ln):
    """x, y, h: FULL saved rows (x only for dres_w, h only with pre_w); st: mean_y, rstd_y, mean_h, rstd_h FULL;
    da, dh FULL (dh may be None).  keep [B, T].  Filtered rows of dx, dy are 0 and add nothing to the sums.
    Returns (grads, mags): mags holds for each gradient the sum of the magnitudes of the terms it is made of."""
    km = np.flatnonzero(np.asarray(keep).reshape(-1))
    seq = km // T
    D = (h if h is not None else y).shape[1]
    pick = lambda v: v[km]  # noqa: E731
    g, mag = {}, {}
    full = lambda v: _full(v, km, B * T)  # noqa: E731
    d = np.zeros((km.size, D)) if dh is None else pick(dh)
    md = np.abs(d)
    if p["pre_w"] is not None:
        hh = (pick(h) - pick(st["mean_h"])[:, None]) * pick(st["rstd_h"])[:, None]
        a = pick(da)
        add, madd = _norm_input_grad(a * p["pre_w"], hh, pick(st["rstd_h"]), ln)
        d, md = d + add, md + madd
        g["dpre_w"], mag["dpre_w"] = np.sum(a * hh, axis=0), np.sum(np.abs(a * hh), axis=0)
        g["dpre_b"], mag["dpre_b"] = np.sum(a, axis=0), np.sum(np.abs(a), axis=0)
    lam = alpha * (1.0 if p["res_w"] is None else p["res_w"])
    g["dx"], mag["dx"] = full(d * lam), full(md * np.abs(lam))
    if p["res_w"] is not None and x is not None:
        g["dres_w"], mag["dres_w"] = alpha * np.sum(d * pick(x), axis=0), abs(alpha) * np.sum(md * np.abs(pick(x)), axis=0)
    if y is None:
        return g, mag
    gt = np.ones((km.size, D)) if p["gate"] is None else np.broadcast_to(p["gate"], (B, D))[seq]
    u, mu = gt * d, np.abs(gt) * md
    if p["post_w"] is not None:
        yh = (pick(y) - pick(st["mean_y"])[:, None]) * pick(st["rstd_y"])[:, None]
        post = yh * p["post_w"] + (0.0 if p["post_b"] is None else p["post_b"])
        dy, _ = _norm_input_grad(u * p["post_w"], yh, pick(st["rstd_y"]), ln)
        _, mdy = _norm_input_grad(mu * np.abs(p["post_w"]), np.abs(yh), pick(st["rstd_y"]), ln)
        g["dpost_w"], mag["dpost_w"] = np.sum(u * yh, axis=0), np.sum(mu * np.abs(yh), axis=0)
        g["dpost_b"], mag["dpost_b"] = np.sum(u, axis=0), np.sum(mu, axis=0)
    else:
        post, dy, mdy = pick(y), u, mu
    g["dy"], mag["dy"] = full(dy), full(mdy)
    if p["gate"] is not None:
        G = p["gate"].shape[0]
        g["dgate"], mag["dgate"] = np.zeros((G, D)), np.zeros((G, D))
        np.add.at(g["dgate"], seq if G > 1 else np.zeros_like(seq), d * post)
        np.add.at(mag["dgate"], seq if G > 1 else np.zeros_like(seq), md * np.abs(post))
    return g, mag


def _full(v, km, M):
    out = np.zeros((M, v.shape[1]))
    out[km] = v
    return out
