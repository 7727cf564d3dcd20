"""The norm of gradients to the last bit where its sums are exact: one rounding to f32, of the root times scale.

And the bound of ordinary sums with that: squares added 16 at a time in f32 (18 2^-24 of the sum, half of it in the
root) and one rounding of the result, 10 2^-24."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

gu = pytest.importorskip("gpu_util")
cl = gu.cl


def norms(t, scale):
    lst = cl.grad_list([t, torch.zeros(3, device=gu.DEV)])
    norm, each = torch.empty(1, device=gu.DEV), torch.empty(2, device=gu.DEV)
    ws = torch.empty(cl.collider_grad_norm_workspace_size(lst, 2), dtype=torch.uint8, device=gu.DEV)
    cl.collider_grad_norm(lst, 2, cl.GRAD_NORM_L2, scale, norm, each, ws)
    cl.collider_check()
    return float(norm), float(each[0])


@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_exact_sums_are_rounded_once(scale):
    """Two values of up to 12 bits in places of different threads: their squares are exact in f32, the sum in f64."""
    r = np.random.default_rng(1)
    scale = float(np.float32(scale))
    t = torch.zeros(9000, device=gu.DEV)
    for a, b in r.integers(1, 4096, size=(300, 2)):
        e = float(2.0 ** r.integers(-20, 20))
        t.zero_()
        t[10], t[4000] = float(a) * e, float(b) * e
        exact = math.sqrt(int(a) ** 2 + int(b) ** 2) * e * scale
        half = float(np.spacing(np.float32(exact))) / 2
        for got in norms(t, scale):
            # (2^-40: what f64 and the correction of the root leave)
            assert abs(got - exact) <= half + exact * 2.0 ** -40, (a, b, e, got, exact)


@pytest.mark.parametrize("n", [1000, 70001, 3000001])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_ordinary_sums(n, dt):
    g = torch.Generator(device=gu.DEV).manual_seed(n)
    t = (torch.randn(n, generator=g, device=gu.DEV) * 0.01).to(dt)
    exact = float(t.double().square().sum().sqrt()) * 0.125
    for got in norms(t, 0.125):
        assert abs(got - exact) <= 10 * 2.0 ** -24 * exact
