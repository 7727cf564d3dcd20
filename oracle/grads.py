"""Norm of a list of gradients and clipping, in float64 (test infrastructure only)."""
from __future__ import annotations

import math

import numpy as np


def norm(grads, kind, scale=1.0):
    """(norm of everything, norm of each), of float64 arrays; a NaN gives NaN.  Largest magnitudes are taken out
    before squaring, so nothing overflows."""
    def one(g):
        g = np.abs(np.asarray(g, np.float64)).reshape(-1)
        big = g.max(initial=0.0) if not np.isnan(g).any() else math.nan
        if kind == "max" or not math.isfinite(big) or big == 0.0:
            return float(big)
        return float(big * math.sqrt(math.fsum((g / big) ** 2)))
    norms = np.array([one(g) for g in grads])
    return (one(norms) if len(norms) else 0.0) * scale, norms * scale


def coefficient(total, max_norm, scale=1.0):
    """What the gradients are multiplied by; 0 (and they are left alone) where the norm, in 32 bits, is not finite."""
    if not math.isfinite(total) or total > float(np.finfo(np.float32).max):
        return 0.0
    return scale * min(1.0, max_norm / (total + 1e-6))
