"""A block's backward over more tokens than a grid is high (65535 blocks of 16 rows of column sums)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

gu = pytest.importorskip("gpu_util")
cl = gu.cl
T, B = 1024, 1100


@pytest.mark.parametrize("arch", [cl.ARCH_LLAMA, cl.ARCH_PHI])
@pytest.mark.parametrize("eight", [False, True])
def test_all_sequences_as_two_halves(arch, eight):
    """Sequences do not meet but in the parameters' gradients: dx of a batch is that of its halves, and the norms'
    gradients are the halves' sums.  Within 2^-6 of dx's largest value (bf16 values on the way may be a step apart where the
    GEMMs are cut elsewhere), and 1e-3 of the gradients' (a million terms of either sign: f32 sums of 8192 additions each
    lose at most 2e-4 of a result a thousand times a term, and steps of bf16 in the terms as much)."""
    llama, D, M = arch == cl.ARCH_LLAMA, 64, B * T
    g = torch.Generator(device=gu.DEV).manual_seed(4)
    n = lambda *s, k=1.0: (torch.randn(*s, generator=g, device=gu.DEV) * k).to(torch.bfloat16)  # noqa: E731
    w = dict(norm1_w=1 + n(D, k=0.1), w_qkv=n(D, 192, k=0.1), w_o=n(64, D, k=0.1), w_up=n(D, 128 if llama else 64, k=0.1),
             w_down=n(64, D, k=0.1))
    t = dict(x=n(M, D), qkv=n(M, 192), o=n(M, 64), up=n(M, 128 if llama else 64))
    f = dict(rstd1=torch.ones(M, device=gu.DEV), lse=torch.full((M,), 8.0, device=gu.DEV))
    if llama:
        w["norm2_w"], t["h"], f["rstd2"] = 1 + n(D, k=0.1), n(M, D), torch.ones(M, device=gu.DEV)
    else:
        t["a"], f["mean1"] = n(M, D), torch.zeros(M, device=gu.DEV)
    dout, keep = n(M, D), (torch.rand(M, generator=g, device=gu.DEV) >= 0.03).to(torch.uint8)
    weights = cl.LayerWeights(**{k: v.data_ptr() for k, v in w.items()})

    def run(b0, b1):
        nb, r = b1 - b0, slice(b0 * T, b1 * T)
        d = cl.LayerDesc(arch=arch, B=nb, T=T, D=D, H=1, Hkv=1, dh=64, F=64, rotary_dim=32, rope_base=1e4, eps=1e-5,
                         norm=cl.NORM_RMS if llama else cl.NORM_LAYER, act=cl.ACT_SWIGLU if llama else cl.ACT_GELU_TANH)
        m = nb * T
        idx, cu, nk = (torch.empty(s, dtype=torch.int32, device=gu.DEV) for s in (m, nb + 1, 1))
        wc = torch.empty(max(cl.collider_compact_workspace_size(nb, T), 1), dtype=torch.uint8, device=gu.DEV)
        cl.collider_compact(keep[r], nb, T, idx, cu, nk, wc)
        new = lambda *s: torch.empty(s, device=gu.DEV)  # noqa: E731
        G = dict(dnorm1_w=new(D), dw_qkv=new(D, 192), dw_o=new(64, D), dw_up=new(*w["w_up"].shape), dw_down=new(64, D))
        G["dnorm2_w" if llama else "dnorm1_b"] = new(D)
        dx = torch.empty(m, D, dtype=torch.bfloat16, device=gu.DEV)
        grads = cl.LayerGrads(dx=dx.data_ptr(), **{k: v.data_ptr() for k, v in G.items()})
        if eight:
            q = {}
            for k, v in t.items():
                c = torch.empty(m, v.shape[1], dtype=torch.uint8, device=gu.DEV)
                e = torch.empty(m, v.shape[1] // 32, dtype=torch.uint8, device=gu.DEV)
                q[k] = cl.ckpt(cl.CKPT_INT8, c, e)
                cl.collider_ckpt_pack(cl.BF16, v[r], v.shape[1], m, v.shape[1], None, None, q[k])
            sv = cl.layer_saved_ckpt(cl.ROWS_FULL, **q, **{k: v[r] for k, v in f.items()})
            ws = torch.empty(cl.collider_layer_ckpt_workspace_size(d), dtype=torch.uint8, device=gu.DEV)
            call = cl.collider_layer_bwd_ckpt
        else:
            sv = cl.LayerSaved(**{k: v[r].data_ptr() for k, v in (*t.items(), *f.items())})
            ws = torch.empty(cl.collider_layer_workspace_size(d), dtype=torch.uint8, device=gu.DEV)
            call = cl.collider_layer_bwd
        call(d, weights, sv, dout[r], cl.ROWS_FULL, idx, cu, nk, grads, cl.ROWS_FULL, ws)
        cl.collider_check()
        return int(nk.item()), dx, G
    kept, dx, G = run(0, B)
    assert kept > 65535 * 16
    (k0, dx0, G0), (k1, dx1, G1) = run(0, B // 2), run(B // 2, B)
    assert k0 + k1 == kept
    halves = torch.cat([dx0, dx1]).float()
    assert float((dx.float() - halves).abs().max()) <= 2.0 ** -6 * float(halves.abs().max())
    for k in ("dnorm1_w", "dnorm2_w" if llama else "dnorm1_b"):
        want = G0[k] + G1[k]
        assert float((G[k] - want).abs().max()) <= 1e-3 * float(want.abs().max()), k
