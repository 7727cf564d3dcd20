"""Where the outputs of the linear backward from a checkpoint may lie.  dX's filtered rows are zeroed while dY's kept rows
are gathered and X is decoded, so a FULL dX may take the place of a FULL dY only row for row, and dX never that of X.
Host checks alone; the addresses are never dereferenced."""
import pytest
import torch

import sparse_backward_gemm_gb300 as cl

FAKE = 1 << 20
WS, X, EXPS, W, IDX, DY, DX, DW = (FAKE * (16 + 4 * i) for i in range(8))
FULL, COMPACT = cl.ROWS_FULL, cl.ROWS_COMPACT


@pytest.fixture(scope="module", autouse=True)
def built():
    from sparse_backward_gemm_gb300 import build
    build.build()


def call(M=64, K=256, N=64, x=X, exps=EXPS, dy=DY, dy_rows=FULL, dx=DX, dx_rows=FULL, dw=DW):
    """The error of a call with a workspace, which without an alias first fails for want of a GPU (or of real memory)."""
    q = cl.Ckpt(format=cl.CKPT_E4M3, code=x, exps=exps, code_ld=256, exp_ld=8)
    status = cl.lib().collider_linear_bwd_ckpt(M, K, N, q, FULL, W, dy, dy_rows, IDX, IDX + 4096, dx, dx_rows, dw, None, WS,
                                               cl.collider_linear_ckpt_workspace_size(M, K, N), 0)
    return status, cl.lib().collider_last_error().decode()


def refused(**kw):
    status, text = call(**kw)
    return status == cl.ERR_INVALID_ARG and "alias" in text


@pytest.mark.parametrize("K,N", [(256, 64), (64, 256), (256, 264)])
def test_full_dx_over_full_dy_of_another_width(K, N):
    assert refused(K=K, N=N, dx=DY)
    assert refused(K=K, N=N, dx=DY, dw=None)


def test_full_dx_across_dy():
    row = 256 * 2
    assert refused(K=256, N=256, dx=DY + row) and refused(K=256, N=256, dx=DY - row)       # not row for row
    assert refused(K=256, N=64, dx=DY - 16) and refused(K=256, N=64, dx=DY + 64 * 64 * 2 - 16)
    assert refused(K=256, N=64, dx=DY - 64 * row + 16, dy_rows=COMPACT)                     # dY's first row is in dX


def test_dx_over_x():
    assert refused(dx=X) and refused(dx=X - 64) and refused(dx=EXPS) and refused(dx=X, dx_rows=COMPACT)


def test_what_may_lie_where():
    row = 256 * 2
    for kw in (dict(), dict(K=256, N=256, dx=DY), dict(K=256, N=64, dx=DY, dx_rows=COMPACT),
               dict(K=256, N=64, dx=DY, dx_rows=COMPACT, dy_rows=COMPACT), dict(K=256, N=64, dx=DY - 64 * row),
               dict(K=256, N=64, dx=DY + 64 * 64 * 2), dict(dx=X, dw=None), dict(dx=None, dw=DW)):
        assert not refused(**kw), kw


@pytest.mark.gpu
@pytest.mark.parametrize("K,N", [(256, 64), (64, 256)])
@pytest.mark.parametrize("dy_rows", [FULL, COMPACT])
def test_compact_dx_over_dy_of_another_width(K, N, dy_rows):
    """COMPACT rows of dX are written after dY's are gathered: the same bits as apart from it."""
    dev, M = "cuda:0", 300
    g = torch.Generator(device=dev).manual_seed(3)
    rows = torch.nonzero(torch.rand(M, generator=g, device=dev) < 0.6).flatten().to(torch.int32)
    idx, nk = torch.cat([rows, rows.new_full((M - rows.numel(),), -1)]), rows.new_tensor([rows.numel()])
    x = torch.randn(M, K, generator=g, device=dev).to(torch.bfloat16)
    q = cl.ckpt(cl.CKPT_INT8, torch.empty(M, K, dtype=torch.uint8, device=dev),
                torch.empty(M, K // 32, dtype=torch.uint8, device=dev))
    cl.collider_ckpt_pack(cl.BF16, x, K, M, K, None, None, q)
    w = torch.randn(K, N, generator=g, device=dev).to(torch.bfloat16)
    dy = torch.randn(M, N, generator=g, device=dev).to(torch.bfloat16)
    ws = torch.empty(cl.collider_linear_ckpt_workspace_size(M, K, N), dtype=torch.uint8, device=dev)
    n = min(-(-rows.numel() // 128) * 128, M)
    got = []
    for apart in (True, False):
        buf = torch.zeros(M * max(K, N), dtype=torch.bfloat16, device=dev)
        buf[: M * N] = dy.flatten()
        dx = torch.empty(M, K, dtype=torch.bfloat16, device=dev) if apart else buf[: M * K].view(M, K)
        dw, db = torch.empty(K, N, device=dev), torch.empty(N, device=dev)
        cl.collider_linear_bwd_ckpt(M, K, N, q, FULL, w, buf, dy_rows, idx, nk, dx, COMPACT, dw, db, ws)
        cl.collider_check()
        got.append((dx[:n].clone(), dw, db))
    for a, b in zip(*got):
        assert torch.equal(a, b)
