"""The residual-join oracle against float64 autograd and finite differences of its own forward."""
import numpy as np
import pytest
import torch

from oracle import join


def _case(ln, gate, res, post=True, pre=True, B=2, T=5, D=16, seed=0):
    rng = np.random.default_rng(seed)
    n = lambda *s: rng.normal(size=s)  # noqa: E731
    p = dict(post_w=1 + 0.2 * n(D) if post else None, post_b=0.3 * n(D) if post and ln else None,
             gate=None if gate == 0 else 0.5 + 0.2 * n(gate, D), res_w=1 + 0.1 * n(D) if res else None,
             pre_w=1 + 0.2 * n(D) if pre else None, pre_b=0.3 * n(D) if pre and ln else None)
    M = B * T
    keep = (rng.random((B, T)) < 0.6).astype(np.uint8)
    keep[0, 0] = 1
    return p, n(M, D), n(M, D), n(M, D), n(M, D), keep, B, T


@pytest.mark.parametrize("ln", [False, True])
@pytest.mark.parametrize("gate", [0, 1, 2])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
def test_backward_is_the_gradient(ln, gate, res, post, pre):
    p, x, y, ga, gh, keep, B, T = _case(ln, gate, res, post, pre)
    alpha, eps = 0.75, 1e-3
    f = join.join_forward(x, y, p, B, T, alpha, ln, eps)
    st = {k: f.get(k) for k in ("mean_y", "rstd_y", "mean_h", "rstd_h")}
    g, _ = join.join_backward(x, y, f["h"], st, ga if pre else None, gh, p, B, T, keep, alpha, ln)

    # autograd of a forward written with torch, the loss over kept rows
    tp = {k: None if v is None else torch.tensor(v, requires_grad=True) for k, v in p.items()}
    tx, ty = torch.tensor(x, requires_grad=True), torch.tensor(y, requires_grad=True)

    def tnorm(v, w, b):
        if ln:
            return torch.nn.functional.layer_norm(v, (v.shape[1],), w, b, eps)
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + eps) * w
    branch = tnorm(ty, tp["post_w"], tp["post_b"]) if post else ty
    if tp["gate"] is not None:
        gt = tp["gate"] if gate > 1 else tp["gate"].expand(B, -1)
        branch = branch * gt.repeat_interleave(T, 0)
    h = alpha * (tx if tp["res_w"] is None else tx * tp["res_w"]) + branch
    km = torch.tensor(keep.reshape(-1) != 0)
    loss = (h * torch.tensor(gh))[km].sum()
    if pre:
        loss = loss + (tnorm(h, tp["pre_w"], tp["pre_b"]) * torch.tensor(ga))[km].sum()
    loss.backward()
    want = dict(dx=tx.grad, dy=ty.grad, dpost_w=tp["post_w"], dpost_b=tp["post_b"], dgate=tp["gate"],
                dres_w=tp["res_w"], dpre_w=tp["pre_w"], dpre_b=tp["pre_b"])
    for k, t in want.items():
        if t is None:
            continue
        t = t if k in ("dx", "dy") else t.grad
        assert np.allclose(g[k], t.numpy(), rtol=1e-10, atol=1e-11), k


def test_forward_and_one_gradient_by_differences():
    p, x, y, ga, gh, keep, B, T = _case(True, 2, True)
    keep[:] = 1
    alpha, eps = 1.25, 1e-3

    def loss(**kw):
        q = dict(p, **{k: v for k, v in kw.items() if k in p})
        f = join.join_forward(kw.get("x", x), kw.get("y", y), q, B, T, alpha, True, eps)
        return np.sum(f["a"] * ga) + np.sum(f["h"] * gh)
    f = join.join_forward(x, y, p, B, T, alpha, True, eps)
    g, _ = join.join_backward(x, y, f["h"], f, ga, gh, p, B, T, keep, alpha, True)
    for name, base, grad in (("x", x, g["dx"]), ("y", y, g["dy"]), ("gate", p["gate"], g["dgate"]),
                             ("res_w", p["res_w"], g["dres_w"]), ("post_b", p["post_b"], g["dpost_b"])):
        rng = np.random.default_rng(5)
        v = rng.normal(size=base.shape)
        d = 1e-6
        fd = (loss(**{name: base + d * v}) - loss(**{name: base - d * v})) / (2 * d)
        assert abs(fd - np.sum(grad * v)) <= 1e-6 * max(1.0, abs(fd)), name


def test_without_a_branch():
    p, x, _, ga, gh, keep, B, T = _case(False, 0, False, post=False)
    f = join.join_forward(x, None, p, B, T, 1.0, False, 1e-3)
    assert "h" not in f
    g, _ = join.join_backward(None, None, x, f, ga, gh, p, B, T, keep, 1.0, False)
    assert set(g) == {"dpre_w", "dpre_b", "dx"}
    tx = torch.tensor(x, requires_grad=True)
    a = tx / torch.sqrt((tx * tx).mean(1, keepdim=True) + 1e-3) * torch.tensor(p["pre_w"])
    km = torch.tensor(keep.reshape(-1) != 0)
    ((a * torch.tensor(ga))[km].sum() + (tx * torch.tensor(gh))[km].sum()).backward()
    assert np.allclose(g["dx"], tx.grad.numpy(), rtol=1e-10, atol=1e-12)
