"""Column sums over more rows than a grid is high (65535 blocks of 16 rows)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

gu = pytest.importorskip("gpu_util")
cl = gu.cl
M = 65536 * 16 + 5 * 16 + 3


def index(n, g, f=0.03):
    rows = torch.nonzero(torch.rand(n, generator=g, device=gu.DEV) >= f).flatten().to(torch.int32)
    return rows, torch.cat([rows, rows.new_full((n - rows.numel(),), -1)]), rows.new_tensor([rows.numel()])


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("dense", [False, True])
def test_linear_bias_gradient(ckpt, dense):
    K, N = 32, 8
    g = torch.Generator(device=gu.DEV).manual_seed(2)
    rows, idx, nk = index(M, g, 0.0 if dense else 0.03)
    assert (rows.numel() == M) == dense
    x = torch.randn(M, K, generator=g, device=gu.DEV).to(torch.bfloat16)
    w = torch.randn(K, N, generator=g, device=gu.DEV).to(torch.bfloat16)
    # whole numbers whose sums stay below 2^24: f32 adds them exactly in any order
    dy = torch.randint(-8, 9, (M, N), generator=g, device=gu.DEV).to(torch.bfloat16)
    dy[-1] = 8
    db = torch.full((N,), 7.0, device=gu.DEV)
    if ckpt:
        q = cl.ckpt(cl.CKPT_INT8, torch.empty(M, K, dtype=torch.uint8, device=gu.DEV),
                    torch.empty(M, 1, dtype=torch.uint8, device=gu.DEV))
        cl.collider_ckpt_pack(cl.BF16, x, K, M, K, None, None, q)
        ws = torch.empty(cl.collider_linear_ckpt_workspace_size(M, K, N), dtype=torch.uint8, device=gu.DEV).fill_(255)
        dw = torch.empty(K, N, device=gu.DEV)
        dx = torch.empty(M, K, dtype=torch.bfloat16, device=gu.DEV)
        cl.collider_linear_bwd_ckpt(M, K, N, q, 0, w, dy, 0, idx, nk, dx, 0, dw, db, ws)
    else:
        ws = torch.empty(cl.collider_linear_workspace_size(cl.BF16, M, K, N), dtype=torch.uint8, device=gu.DEV).fill_(255)
        cl.collider_linear_bwd(cl.BF16, M, K, N, None, 0, None, dy, 0, idx, nk, None, 0, None, db, ws)
    cl.collider_check()
    assert torch.equal(db.double(), dy[rows.long()].double().sum(0))
