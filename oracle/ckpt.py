"""8-bit activation checkpoints in float64: the format include/collider.h states for ``collider_ckpt``, written
with explicit arithmetic (test infrastructure only).

A group is 32 consecutive values of a row.  Its exponent is the smallest e >= -120 with max|v| <= L 2^e (L = 448
for e4m3, 127 for int8), for int8 121 at most; a code is v 2^-e rounded to the nearest representable value, ties to
even, but none whose value would be 2^128: there the largest that decodes to a finite value (240 under e = 120 for
e4m3, 127 under e = 121 for int8).  The byte is e + 127.  A group with a NaN or an infinity: byte 255, codes 0,
decodes to NaN.
"""
from __future__ import annotations

import numpy as np

GROUP = 32
E_MIN = -120
LIMIT = {"e4m3": 448.0, "int8": 127.0}
E_TOP = {"e4m3": 120, "int8": 121}       # the largest exponent, and
TOP_CODE = {"e4m3": 240.0, "int8": 127.0}   # the largest code under it


def e4m3_round(q):
    """Nearest e4m3 value (ties to even) of |q| <= 448: 3 bits behind the leading one, steps of 2^-9 below 2^-6."""
    q = np.asarray(q, dtype=np.float64)
    _, e = np.frexp(q)                                   # q = m 2^e, m in [1/2, 1)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.rint(q / step) * step


def e4m3_code(v):
    """The byte of an e4m3 value."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    _, e = np.frexp(a)
    e = np.maximum(e - 1, -6)                            # exponent of the binade
    mant = np.rint(a / np.ldexp(1.0, e - 3)).astype(np.int64)   # 8..15, below 2^-6: 0..7
    code = np.where(mant >= 8, ((e + 7) << 3) | (mant & 7), mant)
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def e4m3_value(code):
    c = np.asarray(code).astype(np.int64)
    field, frac = (c >> 3) & 15, c & 7
    mag = np.where(field == 0, np.ldexp(frac.astype(np.float64), -9),
                   np.ldexp((8 + frac).astype(np.float64), field - 10))
    mag = np.where((c & 127) == 127, np.nan, mag)
    return np.where(c >= 128, -mag, mag)


def pack(v, fmt):
    """[rows, N] -> (code u8 [rows, N], exps u8 [rows, N / 32])."""
    v = np.asarray(v, dtype=np.float64)
    rows, N = v.shape
    g = v.reshape(rows, N // GROUP, GROUP)
    big = np.max(np.abs(g), axis=2)
    fine = np.isfinite(big)
    big = np.where(fine, big, 0.0)
    m, e = np.frexp(big / LIMIT[fmt])                    # the quotient is m 2^e: a power of two exactly when m = 1/2
    e = np.maximum(np.where(m > 0.5, e, e - 1), E_MIN)
    e = np.minimum(np.where(big > 0, e, E_MIN), E_TOP[fmt])
    q = np.where(fine[..., None], g, 0.0) * np.ldexp(1.0, -e)[..., None]
    lim = np.where(e == E_TOP[fmt], TOP_CODE[fmt], np.inf)[..., None]
    q = np.clip(q, -lim, lim)
    code = e4m3_code(e4m3_round(q)) if fmt == "e4m3" else np.rint(q).astype(np.int8).view(np.uint8)
    return code.reshape(rows, N), np.where(fine, e + 127, 255).astype(np.uint8)


def unpack(code, exps, fmt):
    code, exps = np.asarray(code), np.asarray(exps).astype(np.int64)
    val = e4m3_value(code) if fmt == "e4m3" else code.view(np.int8).astype(np.float64)
    scale = np.where(exps == 255, np.nan, np.ldexp(1.0, np.where(exps == 255, 0, exps) - 127))
    return val * np.repeat(scale, GROUP, axis=1)
