"""Weight gradients of the feed-forward block take at most 2^27 tokens: one pair of SMs may have to add all of them, 64
in up to 0.3 us, and its epilogue waits 2 s for that at most."""
import pytest

import sparse_backward_gemm_gb300 as cl

MB, GB = 1 << 20, 1 << 40
LIMIT = 1 << 27


@pytest.fixture(scope="module", autouse=True)
def built():
    from sparse_backward_gemm_gb300 import build
    build.build()


def call(M, dx=True, dw_up=True, dw_down=True, idx=None, nk=None):
    d = cl.FfnDesc(M=M, D=8, F=8, act=cl.GLU_SILU, grad_dtype=cl.F32)
    with pytest.raises(cl.ColliderError) as e:
        cl.collider_ffn_bwd(d, MB, 2 * MB, GB, 2 * GB, 0, 3 * GB, 0, idx, nk, 4 * GB if dx else None, 0, 3 * MB if dw_up else None,
                            4 * MB if dw_down else None, None, stream=0)
    return e.value.status, str(e.value)


@pytest.mark.parametrize("wanted", [dict(), dict(dw_up=False), dict(dw_down=False), dict(dx=False), dict(idx=5 * MB, nk=6 * MB)])
def test_more_tokens_are_refused(wanted):
    for M in (LIMIT + 1, 1 << 30):
        status, text = call(M, **wanted)
        assert status == cl.ERR_UNSUPPORTED and "2^27 tokens" in text, text
    status, text = call(LIMIT, **wanted)
    assert status == cl.ERR_INVALID_ARG and "workspace" in text, text


def test_without_weight_gradients_they_are_taken():
    status, text = call(1 << 30, dw_up=False, dw_down=False)
    assert status == cl.ERR_INVALID_ARG and "workspace" in text, text
    d = cl.FfnDesc(M=1 << 30, D=8, F=8, act=cl.GLU_SILU, grad_dtype=cl.F32)
    assert cl.collider_ffn_fwd_workspace_size(d) > 0 and cl.collider_ffn_bwd_workspace_size(d) > 0


@pytest.mark.gpu
@pytest.mark.parametrize("with_dx", [True, False])
def test_as_many_as_are_taken(with_dx):
    """2^27 tokens, all but a few of them with dy = 0: sums of small whole numbers, exact in every order."""
    torch = pytest.importorskip("torch")
    dev, bf, M, D, F = "cuda:0", torch.bfloat16, LIMIT, 8, 8
    x, dy = torch.ones(M, D, dtype=bf, device=dev), torch.zeros(M, D, dtype=bf, device=dev)
    up = torch.zeros(M, 2 * F, dtype=bf, device=dev)
    up[:, F:] = 1.0                                    # g = 0, u = 1: act 0, its slope 1/2
    at = torch.tensor([0, 1, 63, 64, M // 2, M - 65, M - 64, M - 1], device=dev)
    dy[at, 0] = 2.0
    w_up = torch.ones(D, 2 * F, dtype=bf, device=dev)
    w_down = torch.eye(F, dtype=bf, device=dev)        # ds = dy
    dx = torch.full((M, D), 7.0, dtype=bf, device=dev) if with_dx else None
    dw_up, dw_down = torch.full((D, 2 * F), 7.0, device=dev), torch.full((F, D), 7.0, device=dev)
    d = cl.FfnDesc(M=M, D=D, F=F, act=cl.GLU_SILU, grad_dtype=cl.F32)
    ws = torch.empty(cl.collider_ffn_bwd_workspace_size(d), dtype=torch.uint8, device=dev)
    cl.collider_ffn_bwd(d, w_up, w_down, x, up, 0, dy, 0, None, None, dx, 0, dw_up, dw_down, ws)
    cl.collider_check()
    want = torch.zeros(D, 2 * F, device=dev)
    want[:, 0] = float(at.numel())                     # dg = 2 . 1 . 1/2 of one column in each of the rows
    assert torch.equal(dw_up, want) and not dw_down.any()
    if with_dx:
        assert bool((dx[at] == 1.0).all()) and int(dx.count_nonzero()) == at.numel() * D
