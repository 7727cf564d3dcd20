"""A kept index outside the tokens in the stack's backward: reported, nothing read through it, and the embedding
gradients of ids that only other sequences hold as they are without it."""
import numpy as np
import pytest
import torch

import workloads
from oracle import stack as ost

pytestmark = pytest.mark.gpu

gu = pytest.importorskip("gpu_util")
cl = gu.cl


@pytest.mark.parametrize("bad", [2 ** 31 - 1, 2 * 192, -1])
def test_stack(bad):
    ls = workloads.LayerShape(seed_base=87000, arch="llama", B=2, T=192, D=256, H=4, Hkv=2, dh=64, F=384, rotary_dim=64,
                              rope_base=10000.0, norm="rms", eps=1e-5, act="swiglu", qkv_bias=False, out_bias=False,
                              mlp_bias=False, f=0.4, mask="gumbel")
    st = workloads.StackShape(seed_base=86000, layer=ls, L=2, V=512)
    t = workloads.stack_tensors(st)
    z, saved = ost.stack_forward(t["ids"], t["E"], t["layers"], t["normf_w"], t["w_lm"], ls, round_saved=True)
    layers = [gu.DeviceLayer(ls, t["layers"][l], saved["blocks"][l]) for l in range(st.L)]
    W = (cl.LayerWeights * st.L)(*[L.weights for L in layers])
    S = (cl.LayerSaved * st.L)(*[L.saved for L in layers])
    G = (cl.LayerGrads * st.L)(*[L.grads for L in layers])
    D, V = ls.D, st.V
    desc = gu.layer_desc(ls)
    ws = torch.zeros(cl.collider_stack_workspace_size(desc, st.L, V), dtype=torch.uint8, device=gu.DEV)
    ins = [gu.bf16(z), gu.i32(t["targets"]), gu.i32(t["ids"]), gu.bf16(saved["y"]), gu.bf16(saved["xL"]),
           gu.f32(saved["rstdf"]), gu.bf16(t["normf_w"]), gu.bf16(t["w_lm"])]
    idx, cu, nk = gu.compact(t["keep"])

    def run(index):
        dnf, dlm, dE = (torch.full(shp, float("nan"), device=gu.DEV) for shp in ((D,), (D, V), (V, D)))
        cl.collider_stack_bwd(desc, st.L, V, W, S, *ins, index, cu, nk, G, dnf, dlm, dE, ws)
        torch.cuda.synchronize()
        return dE
    want = run(idx)
    cl.collider_check()
    index = idx.clone()
    index[int(nk.item()) - 1] = bad
    got = run(index)
    with pytest.raises(cl.ColliderError) as e:
        cl.collider_check()
    assert e.value.status == cl.ERR_INVALID_ARG and "index outside its buffer" in str(e.value)
    ids = np.asarray(t["ids"]).reshape(ls.B, ls.T)
    elsewhere = np.setdiff1d(np.arange(V), ids[1])
    assert np.intersect1d(elsewhere, ids[0]).size > 20
    at = torch.from_numpy(elsewhere).to(gu.DEV)
    assert torch.equal(got[at], want[at])
    assert torch.equal(run(idx), want)
    cl.collider_check()
