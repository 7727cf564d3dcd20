"""The feed-forward backward at gates that bf16 holds and training hardly meets: the activation's slope there is 1 or 0.

Bounds as in test_gpu_ffn.py, but from |g| = 150 on the activation is the gate itself or 0 and its slope 1 or 0, in f32
too (e^-150 is below its smallest value): nothing but the f32 sum of ds and the roundings to bf16 is lost there."""
import numpy as np
import pytest

import test_gpu_ffn as t
from oracle import ffn as off

pytestmark = pytest.mark.gpu

H, E = t.H, t.E
FAR = 150.0


def bounds(v, kind):
    o = off.backward(v["x"], v["up"], v["dy"], v["w_up"], v["w_down"], kind)
    x, up, dy = (np.abs(v[k]) for k in ("x", "up", "dy"))
    D, F, n = x.shape[1], v["w_down"].shape[0], x.shape[0]
    g, u = np.split(up, 2, axis=1)
    a, da = (np.abs(w) for w in off.act(np.split(v["up"], 2, axis=1)[0], kind))
    wd, wu = np.abs(v["w_down"]), np.abs(v["w_up"])
    mag, near = dy @ wd.T, np.where(g < FAR, 2.0 ** -18 * (1 + g), 0.0)
    # f32 products: two more roundings each
    e_dup = np.concatenate((mag * u * (da * E(D + 4) + 1.2 * near), mag * (a * E(D + 4) + g * near)), axis=1)
    e_dup = e_dup + H * (np.abs(o["dup"]) + e_dup)
    e_s = u * (a * E(4) + g * near)
    e_s = e_s + H * (np.abs(o["s"]) + e_s)
    dup, s = np.abs(o["dup"]) + e_dup, np.abs(o["s"]) + e_s
    ex = e_dup @ wu.T + E(2 * F) * (dup @ wu.T)
    eu = x.T @ e_dup + E(n) * (x.T @ dup)
    ed = e_s.T @ dy + E(n) * (s.T @ dy)
    return o, dict(dx=ex + H * (np.abs(o["dx"]) + ex), dw_up=eu + H * (np.abs(o["dw_up"]) + eu),
                   dw_down=ed + H * (np.abs(o["dw_down"]) + ed))


def check(v, kind):
    got = t.run_backward(v, kind, None, None, None)
    o, b = bounds(v, kind)
    for name, w in zip(("dx", "dw_up", "dw_down"), got):
        t.within(w, o[name], b[name], name)


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("far", [1e3, 1e7, 1e13, 1e18, 3e19, 5e19, 1e20, 1e25, 3e38])
def test_far_gates(kind, far):
    """Gates of +-far in two hidden columns, whose up projections weigh nothing in dx."""
    M, D, F = 140, 72, 136
    v = t.inputs(M, D, F, 31)
    far = float(t.workloads.bf16_representable(np.float32(far)))
    v["up"][3::7, 5], v["up"][4::7, 5], v["up"][5::7, 129], v["up"][6::7, 129] = far, -far, far, -far
    v["up"][:, F + 5] *= 2.0 ** -8               # (so that s = g u stays inside bf16)
    v["up"][:, F + 129] *= 2.0 ** -8
    v["dy"] *= 2.0 ** -10                        # (and du = ds g)
    v["w_up"][:, F + 5] = v["w_up"][:, F + 129] = 0.0
    check(v, kind)


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_a_slope_of_0_beside_a_large_product(kind):
    """ds u beyond f32 where the slope is 0: the gate's gradient is 0, not 0 times infinity."""
    M, D, F = 20, 64, 64
    v = t.inputs(M, D, F, 32)
    big = 2.0 ** 70
    v["dy"][7] *= big
    v["up"][7, 9], v["up"][7, F + 9] = -200.0, big
    check(v, kind)
