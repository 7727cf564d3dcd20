"""Up to 64 tokens the forward keeps s as the sum of two bf16 values, whatever the weights' sizes: y is off by its own
rounding and by H of H of s (test_gpu_ffn.py counts H of s from 33 tokens on)."""
import numpy as np
import pytest

import test_gpu_ffn as t
from oracle import ffn as off

pytestmark = pytest.mark.gpu

H, E = t.H, t.E


def bound(v, kind):
    o = off.forward(v["x"], v["w_up"], v["w_down"], kind)
    D, F = v["x"].shape[1], v["w_down"].shape[0]
    e_up = E(D) * (np.abs(v["x"]) @ np.abs(v["w_up"]))
    g, u = np.split(np.abs(o["up"]), 2, axis=1)
    eg, eu = np.split(e_up, 2, axis=1)
    ds = 1.2 * eg * (u + eu) + g * eu + 2.0 ** -18 * (1 + g) * g * u      # |a'| < 1.2, |a| <= |g|
    ds = ds + H * H * (np.abs(o["s"]) + ds)
    wd = np.abs(v["w_down"])
    ey = ds @ wd + E(2 * F) * ((np.abs(o["s"]) + ds) @ wd)                # (two products a value of s)
    return o, H * (np.abs(o["y"]) + ey) + ey


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,D,F", [(33, 256, 384), (33, 8, 8), (48, 256, 384), (64, 64, 64), (64, 256, 384), (57, 520, 136),
                                   (33, 1536, 96), (40, 520, 1032), (64, 2048, 264), (32, 256, 384), (7, 256, 384)])
def test_two_values_of_s(M, D, F, kind):
    v = t.inputs(M, D, F, M + D + F)
    o, b = bound(v, kind)
    up, y = t.run_forward(v, kind)
    t.within(y, o["y"], b, "y")
    up2, y2 = t.run_forward(v, kind, (8, 24, 16))
    assert t.torch.equal(up2, up) and t.torch.equal(y2, y)
