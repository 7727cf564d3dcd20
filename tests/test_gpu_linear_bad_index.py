"""A kept index outside the rows in the f32 linear backward: its row counts as zeros and is written nowhere, the index is
reported, and the other rows' results stand."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

gu = pytest.importorskip("gpu_util")
cl = gu.cl


@pytest.mark.parametrize("bad", [200, 2 ** 31 - 1, -3, -(2 ** 31)])
@pytest.mark.parametrize("only_db", [False, True])
def test_f32(bad, only_db):
    M, K, N = 200, 72, 64
    rng = np.random.default_rng(6)
    X, W, dY = (gu.f32(rng.normal(size=s)) for s in ((M, K), (K, N), (M, N)))
    idx = np.arange(M)
    idx[33] = bad
    ws = torch.zeros(cl.collider_linear_workspace_size(cl.F32, M, K, N), dtype=torch.uint8, device=gu.DEV)
    dX, dW, db = torch.full((M, K), 7.0, device=gu.DEV), torch.empty(K, N, device=gu.DEV), torch.empty(N, device=gu.DEV)
    if only_db:
        cl.collider_linear_bwd(cl.F32, M, K, N, None, 0, None, dY, 0, gu.i32(idx), gu.i32([M]), None, 0, None, db, ws)
    else:
        cl.collider_linear_bwd(cl.F32, M, K, N, X, 0, W, dY, 0, gu.i32(idx), gu.i32([M]), dX, 0, dW, db, ws)
    with pytest.raises(cl.ColliderError) as e:
        cl.collider_check()
    assert e.value.status == cl.ERR_INVALID_ARG and "index outside its buffer" in str(e.value)
    x, g = gu.host(X), gu.host(dY)
    x[33] = g[33] = 0
    # f32 sums of M (or N) products: each addition and product within 2^-24 of the magnitudes so far
    assert np.all(np.abs(gu.host(db) - g.sum(0)) <= (M + 1) * 2.0 ** -24 * np.abs(g).sum(0))
    if not only_db:
        assert np.all(np.abs(gu.host(dW) - x.T @ g) <= (M + 1) * 2.0 ** -24 * (np.abs(x).T @ np.abs(g)))
        w = gu.host(W)
        assert np.all(np.abs(gu.host(dX) - g @ w.T) <= (N + 1) * 2.0 ** -24 * (np.abs(g) @ np.abs(w).T))
    cl.collider_check()
