"""The 8-bit checkpoint oracle at the top of the range: every finite value is kept finite, within what the format
promises."""
import numpy as np
import pytest

from oracle import ckpt

TOP = float(np.finfo(np.float32).max)
BF_TOP = (2.0 - 2.0 ** -7) * 2.0 ** 127


def largest():
    """Groups whose largest value is one of the last steps below 2^128, beside smaller ones of both signs."""
    big = [TOP, BF_TOP, 3.3e38, 3.38e38, 127.0 * 2.0 ** 121, 127.5 * 2.0 ** 121, 248.0 * 2.0 ** 120, 247.5 * 2.0 ** 120,
           240.0 * 2.0 ** 120, 224.0 * 2.0 ** 120, 2.0 ** 127, 126.5 * 2.0 ** 121, 63.5 * 2.0 ** 121]
    v = np.zeros((2 * len(big), 32))
    for i, b in enumerate(big):
        v[2 * i], v[2 * i + 1] = np.linspace(-b, b, 32), np.where(np.arange(32) % 3 == 0, b, 2.0 ** 119)
    return v.astype(np.float32).astype(np.float64)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_finite_values_stay_finite_and_near(fmt):
    v = largest()
    code, exps = ckpt.pack(v, fmt)
    back = ckpt.unpack(code, exps, fmt)
    assert np.all(np.abs(back) <= TOP)
    off = np.abs(back - v)
    e = np.repeat(exps.astype(np.int64) - 127, 32, axis=1)
    if fmt == "e4m3":
        assert e.max() <= 120 and np.all(off <= np.maximum(2.0 ** -4 * np.abs(v), np.ldexp(1.0, e - 10)))
    else:
        past = np.abs(v) > 127.5 * 2.0 ** 121          # kept as 127 * 2^121
        assert e.max() == 121 and past.any() and np.all(off[~past] <= np.ldexp(1.0, e - 1)[~past])
        assert np.all(off[past] < 2.0 ** 121) and np.all(np.abs(back[past]) == 127 * 2.0 ** 121)
        assert np.all(code.view(np.int8) >= -127)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_below_the_top_nothing_changes(fmt):
    """The largest values that need no clamp: 247.5 * 2^120 rounds to 240 * 2^120, 127 * 2^121 is a code of its own."""
    v = np.zeros((1, 32))
    v[0, 0] = 247.5 * 2.0 ** 120 if fmt == "e4m3" else 127.0 * 2.0 ** 121
    want = 240.0 * 2.0 ** 120 if fmt == "e4m3" else 127.0 * 2.0 ** 121
    assert ckpt.unpack(*ckpt.pack(v, fmt), fmt)[0, 0] == want
