"""A kept index outside the tokens in the attention's and a block's backward: no read or write beyond a buffer, the index
reported, and the sequences it is not in as they are without it.  (The parameters' gradients of such a call are not
defined.)"""
import pytest
import torch

import workloads
from test_gpu_layer_ckpt import case, given

pytestmark = pytest.mark.gpu

gu = pytest.importorskip("gpu_util")
cl = gu.cl


def spoiled(s, idx, nk, bad):
    """The index list with the last kept token of the last sequence replaced, and that token."""
    out, n = idx.clone(), int(nk.item())
    token = int(out[n - 1])
    assert token >= s.M - s.T
    out[n - 1] = bad
    return out, token


def reported():
    with pytest.raises(cl.ColliderError) as e:
        cl.collider_check()
    assert e.value.status == cl.ERR_INVALID_ARG and "index outside its buffer" in str(e.value)
    cl.collider_check()


@pytest.mark.parametrize("bad", ["next", "largest", "negative"])
@pytest.mark.parametrize("name", ["llama", "qwen", "phi"])
@pytest.mark.parametrize("eight", [False, True])
def test_block(name, eight, bad):
    s, w, t, saved, cks = case(name, "e4m3")
    L = gu.DeviceLayer(s, w, saved)
    idx, cu, nk = gu.compact(t["keep"])
    dout = gu.bf16(t["dout"])
    ws = torch.zeros(cl.collider_layer_ckpt_workspace_size(L.desc), dtype=torch.uint8, device=gu.DEV)
    sc = given(s, cks, "e4m3", saved, t["keep"], cl.ROWS_FULL)

    def run(index):
        L.dx.fill_(float("nan"))
        if eight:
            cl.collider_layer_bwd_ckpt(L.desc, L.weights, sc, dout, cl.ROWS_FULL, index, cu, nk, L.grads, cl.ROWS_FULL, ws)
        else:
            cl.collider_layer_bwd(L.desc, L.weights, L.saved, dout, cl.ROWS_FULL, index, cu, nk, L.grads, cl.ROWS_FULL, ws)
        torch.cuda.synchronize()
        return L.dx.clone()
    want = run(idx)
    cl.collider_check()
    index, token = spoiled(s, idx, nk, {"next": s.M, "largest": 2 ** 31 - 1, "negative": -5}[bad])
    got = run(index)
    reported()
    if bad != "negative":      # (an ascending list still: its filtered tokens are found)
        first = slice(0, (s.B - 1) * s.T)
        assert torch.equal(got[first], want[first])
        assert bool((got[token] == 0).all())
    assert torch.equal(run(idx), want)
    cl.collider_check()


@pytest.mark.parametrize("bad", [2 ** 31 - 1, -1, 10 ** 6])
@pytest.mark.parametrize("dh", [64, 128])
def test_attention(dh, bad):
    B, T, H, Hkv = 2, 150, 4, 2
    M = B * T
    g = torch.Generator(device=gu.DEV).manual_seed(dh)
    n = lambda h: torch.randn(M, h * dh, generator=g, device=gu.DEV).to(torch.bfloat16)  # noqa: E731
    q, k, v, o, do = n(H), n(Hkv), n(Hkv), n(H), n(H)
    lse = torch.full((B, H, T), 8.0, device=gu.DEV)
    idx, cu, nk = gu.compact(workloads.gumbel_keep_mask(B, T, 0.4, seed=3))
    ws = torch.zeros(cl.collider_attn_workspace_size(B, T, H, Hkv, dh), dtype=torch.uint8, device=gu.DEV)

    def run(index):
        d = [torch.full_like(t, 7.0) for t in (q, k, v)]
        cl.collider_attn_bwd(B, T, H, Hkv, dh, 1, dh ** -0.5, dh, 1e4, q, k, v, o, do, H * dh, Hkv * dh, H * dh, cl.ROWS_FULL,
                             lse, index, cu, nk, *d, cl.ROWS_FULL, ws)
        torch.cuda.synchronize()
        return d
    want = run(idx)
    cl.collider_check()
    index = idx.clone()
    index[int(nk.item()) - 1] = bad
    got = run(index)
    reported()
    if bad > 0:
        for a, b in zip(got, want):
            assert torch.equal(a[:T], b[:T])
    for a, b in zip(run(idx), want):
        assert torch.equal(a, b)
    cl.collider_check()
