"""The 8-bit checkpoint oracle against what the format promises: exhaustively over the codes, and on values
chosen where rounding and the choice of the exponent can go wrong."""
import numpy as np
import pytest

from oracle import ckpt
import workloads


def test_every_e4m3_code_round_trips():
    codes = np.arange(256, dtype=np.uint8)
    v = ckpt.e4m3_value(codes)
    fine = ~np.isnan(v)
    assert np.array_equal(np.flatnonzero(~fine), [127, 255])
    assert np.nanmax(v) == 448 and np.min(np.abs(v[fine & (v != 0)])) == 2.0 ** -9
    assert np.array_equal(ckpt.e4m3_code(v[fine]), codes[fine])
    assert np.array_equal(ckpt.e4m3_round(v[fine]), v[fine])


def test_e4m3_rounding_is_nearest_even():
    v = np.sort(ckpt.e4m3_value(np.arange(127, dtype=np.uint8)))      # 0 .. 448
    rng = np.random.default_rng(0)
    q = np.concatenate([rng.uniform(0, 448, 4000), rng.uniform(0, 0.1, 4000), (v[1:] + v[:-1]) / 2])
    got = ckpt.e4m3_round(q)
    near = np.abs(q[:, None] - v[None, :])
    assert np.array_equal(np.abs(got - q), near.min(axis=1))
    ties = ckpt.e4m3_code(got[8000:])
    assert np.all(ties % 2 == 0)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_exponent_is_the_smallest_and_values_are_kept(fmt):
    rng = np.random.default_rng(1)
    v = rng.normal(size=(64, 96)) * np.exp(rng.uniform(-40, 40, size=(64, 1)))
    v = workloads.bf16_representable(v).astype(np.float64)
    v[3] = 0.0
    v[4, 0], v[4, 1:32] = 448.0, 1.0            # exactly at a limit, and one bf16 step beyond it
    v[5, 0], v[5, 1:32] = 450.0, 1.0
    v[6, 0], v[6, 1:32] = 127.0, 1.0
    v[7, 0], v[7, 1:32] = 127.5, 1.0
    code, exps = ckpt.pack(v, fmt)
    e = np.repeat(exps.astype(np.int64) - 127, 32, axis=1)
    big = np.repeat(np.abs(v).reshape(64, 3, 32).max(axis=2), 32, axis=1)
    assert np.all(big <= ckpt.LIMIT[fmt] * np.ldexp(1.0, e))
    assert np.all((e == ckpt.E_MIN) | (big > ckpt.LIMIT[fmt] * np.ldexp(1.0, e - 1)))
    back = ckpt.unpack(code, exps, fmt)
    off = np.abs(back - v)
    if fmt == "e4m3":
        assert np.all(off <= np.maximum(2.0 ** -4 * np.abs(v), np.ldexp(1.0, e - 10)))
    else:
        assert np.all(off <= np.ldexp(1.0, e - 1))
    # decoding is exact in bf16
    assert np.array_equal(workloads.bf16_representable(back).astype(np.float64), back)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_non_finite_groups_and_tiny_values(fmt):
    v = np.zeros((4, 64))
    v[0, 5], v[1, 40], v[2, 3] = np.nan, -np.inf, 2.0 ** -126
    v[3, :] = -0.0
    code, exps = ckpt.pack(v, fmt)
    assert exps[0].tolist() == [255, 7] and exps[1].tolist() == [7, 255] and exps[2].tolist() == [7, 7]
    back = ckpt.unpack(code, exps, fmt)
    assert np.all(np.isnan(back[0, :32])) and np.all(back[0, 32:] == 0) and np.all(np.isnan(back[1, 32:]))
    assert back[2, 3] == (2.0 ** -126 if fmt == "e4m3" else 0.0)   # int8 keeps whole multiples of 2^-120
    assert np.all(back[3] == 0)
