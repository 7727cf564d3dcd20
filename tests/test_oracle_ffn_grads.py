"""The gated feed-forward oracle against finite differences and float64 autograd; the gradient norm's against closed
forms."""
import math

import numpy as np
import pytest
import torch

from oracle import ffn, grads


def tensors(seed, M=5, D=7, F=6):
    r = np.random.default_rng(seed)
    return r.normal(size=(M, D)), r.normal(size=(D, 2 * F)), r.normal(size=(F, D)), r.normal(size=(M, D))


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_backward_against_autograd(kind):
    x, wu, wd, dy = tensors(1)
    keep = np.array([1, 0, 1, 1, 0], bool)
    t = [torch.tensor(v, dtype=torch.float64, requires_grad=True) for v in (x, wu, wd)]
    g, u = (t[0] @ t[1]).chunk(2, 1)
    a = torch.nn.functional.silu(g) if kind == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
    y = (a * u) @ t[2]
    f = ffn.forward(x, wu, wd, kind)
    assert np.allclose(f["y"], y.detach().numpy(), rtol=1e-12, atol=1e-12)
    y.backward(torch.tensor(dy * keep[:, None]))
    b = ffn.backward(x, f["up"], dy, wu, wd, kind, keep)
    for k, v in zip(("dx", "dw_up", "dw_down"), t):
        assert np.allclose(b[k], v.grad.numpy(), rtol=1e-11, atol=1e-12), k


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_backward_against_differences(kind):
    x, wu, wd, dy = tensors(2)
    f = lambda x, wu, wd: float((ffn.forward(x, wu, wd, kind)["y"] * dy).sum())  # noqa: E731
    b = ffn.backward(x, ffn.forward(x, wu, wd, kind)["up"], dy, wu, wd, kind)
    r = np.random.default_rng(3)
    for i, k in enumerate(("dx", "dw_up", "dw_down")):
        d = r.normal(size=(x, wu, wd)[i].shape)
        step = [(x, wu, wd)[j] * 0 for j in range(3)]
        step[i] = d * 1e-5
        diff = (f(x + step[0], wu + step[1], wd + step[2]) - f(x - step[0], wu - step[1], wd - step[2])) / 2e-5
        assert math.isclose(diff, float((b[k] * d).sum()), rel_tol=1e-7)


def test_act_far_out():
    for kind in ("silu", "gelu_tanh"):
        a, da = ffn.act([-1000.0, -30.0, 0.0, 30.0, 1000.0], kind)
        assert np.allclose(a, [0, 0, 0, 30, 1000], atol=1e-11) and np.allclose(da, [0, 0, 0.5, 1, 1], atol=1e-11)


def test_filtered_rows_count_for_nothing():
    x, wu, wd, dy = tensors(4)
    up = ffn.forward(x, wu, wd, "silu")["up"]
    keep = np.array([0, 1, 1, 0, 1], bool)
    want = ffn.backward(x[keep], up[keep], dy[keep], wu, wd, "silu")
    for v in (x, up, dy):
        v[~keep] = np.nan
    got = ffn.backward(x, up, dy, wu, wd, "silu", keep)
    assert np.allclose(got["dw_up"], want["dw_up"]) and np.allclose(got["dw_down"], want["dw_down"])
    assert np.allclose(got["dx"][keep], want["dx"]) and not got["dx"][~keep].any()


def test_norms():
    total, each = grads.norm([np.array([3.0, 0.0]), np.array([]), np.array([[-4.0]])], "l2")
    assert total == 5.0 and each.tolist() == [3.0, 0.0, 4.0]
    total, each = grads.norm([np.array([3.0, 0.0]), np.array([[-4.0]])], "max", 0.5)
    assert total == 2.0 and each.tolist() == [1.5, 2.0]
    assert math.isclose(grads.norm([np.full(100, 1e300)], "l2")[0], 1e301)
    assert math.isnan(grads.norm([np.array([1.0, math.nan]), np.array([math.inf])], "l2")[0])
    assert grads.norm([], "l2")[0] == 0.0
    assert grads.coefficient(5.0, 1.0, 2.0) == 2.0 / (5.0 + 1e-6) and grads.coefficient(0.5, 1.0) == 1.0
    assert grads.coefficient(1e39, 1.0) == 0.0 and grads.coefficient(math.nan, 1.0) == 0.0
