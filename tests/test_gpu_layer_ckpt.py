"""A block's backward from a saved set in 8 bits: bit for bit the backward of the decoded saved set, which the
oracle's gradients of those decoded values are compared with."""
import numpy as np
import pytest
import torch

import workloads
from oracle import block as ob
from oracle import ckpt as ock

pytestmark = pytest.mark.gpu

gu = pytest.importorskip("gpu_util")
cl = gu.cl
FMT = {"e4m3": cl.CKPT_E4M3, "int8": cl.CKPT_INT8}

LLAMA = workloads.LayerShape(seed_base=91000, arch="llama", B=2, T=160, D=256, H=4, Hkv=2, dh=64, F=384, rotary_dim=64,
                             rope_base=10000.0, norm="rms", eps=1e-5, act="swiglu", qkv_bias=False, out_bias=False,
                             mlp_bias=False, f=0.4, mask="gumbel")
SHAPES = {
    "llama": LLAMA,
    "qwen": LLAMA.with_(seed_base=92000, T=200, H=2, Hkv=1, dh=128, rotary_dim=128, rope_base=1e6, qkv_bias=True),
    "phi": LLAMA.with_(seed_base=93000, T=150, arch="phi", Hkv=4, rotary_dim=32, norm="ln", act="gelu", qkv_bias=True,
                       out_bias=True, mlp_bias=True, mask="span"),
}


def case(name, fmt, f=None):
    """The block, its inputs, and its saved set with every checkpointed tensor replaced by its decoded values."""
    s = SHAPES[name] if f is None else SHAPES[name].with_(f=f)
    w, t = workloads.layer_weights(s), workloads.layer_inputs(s)
    _, saved = ob.block_forward(t["x"], w, s, round_saved=True)
    up = "gu" if s.arch == "llama" else "f1"
    cks = {}
    for k in ("x", "qkv", "o", up) + (("h",) if s.arch == "llama" else ("a",)):
        v = np.asarray(saved[k], np.float64).reshape(s.M, -1)
        cks["up" if k == up else k] = ock.pack(v, fmt)
        saved[k] = ock.unpack(*ock.pack(v, fmt), fmt).reshape(np.shape(saved[k]))
    return s, w, t, saved, cks


def given(s, cks, fmt, saved, keep, rows, pinned=False):
    km = np.flatnonzero(keep.reshape(-1))
    out = {}
    for k, (c, e) in cks.items():
        if rows == cl.ROWS_COMPACT:
            c, e = c[km], e[km]
        c, e = (torch.from_numpy(np.ascontiguousarray(v)) for v in (c, e))
        c, e = (c.pin_memory(), e.pin_memory()) if pinned else (c.to(gu.DEV), e.to(gu.DEV))
        out[k] = cl.ckpt(FMT[fmt], c, e)
    for k in ("mean1", "rstd1", "lse", "rstd2"):
        if k in saved:
            out[k] = gu.f32(saved[k])
    return cl.layer_saved_ckpt(rows, **out)


@pytest.mark.parametrize("name", ["llama", "qwen", "phi"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("rows,pinned", [(cl.ROWS_FULL, False), (cl.ROWS_COMPACT, False), (cl.ROWS_COMPACT, True)])
def test_block_backward_from_checkpoints(name, fmt, rows, pinned):
    s, w, t, saved, cks = case(name, fmt)
    L = gu.DeviceLayer(s, w, saved)
    if s.arch == "llama":
        L.saved.a = L.saved.b = L.saved.s = None      # recomputed, as from checkpoints
    idx, cu, nk = gu.compact(t["keep"])
    dout = gu.bf16(t["dout"])
    L.run(dout, idx, cu, nk)
    cl.collider_check()
    want = L.results()
    for v in list(L.grads_t.values()) + [L.dx]:
        v.fill_(float("nan"))
    ws = torch.empty(cl.collider_layer_ckpt_workspace_size(L.desc), dtype=torch.uint8, device=gu.DEV).fill_(255)
    sc = given(s, cks, fmt, saved, t["keep"], rows, pinned)
    cl.collider_layer_bwd_ckpt(L.desc, L.weights, sc, dout, cl.ROWS_FULL, idx, cu, nk, L.grads, cl.ROWS_FULL, ws)
    cl.collider_check()
    got = L.results()
    for k in want:
        assert np.array_equal(got[k], want[k]), k
    # the oracle on the decoded saved set (LLAMA: a, b and s of the decoded x, h and up)
    if s.arch == "llama":
        x, h, g = (np.asarray(saved[k], np.float64) for k in ("x", "h", "gu"))
        r = lambda v: workloads.bf16_representable(v).astype(np.float64)  # noqa: E731
        saved["a"] = r(x * np.asarray(saved["rstd1"])[:, None] * w["norm1_w"])
        saved["b"] = r(h * np.asarray(saved["rstd2"])[:, None] * w["norm2_w"])
        gate, up = g[:, :s.F], g[:, s.F:]
        saved["s"] = r(gate / (1 + np.exp(-gate)) * up)
    ref = ob.block_backward(t["dout"], saved, w, s, t["keep"])
    for k in ref:
        assert gu.rel_err(got[k], ref[k]) <= 2e-2, (k, gu.rel_err(got[k], ref[k]))
    assert np.all(got["dx"][t["keep"].reshape(-1) == 0] == 0)


def test_nothing_kept_and_a_captured_call():
    s, w, t, saved, cks = case("llama", "e4m3")
    L = gu.DeviceLayer(s, w, saved)
    ws = torch.empty(cl.collider_layer_ckpt_workspace_size(L.desc), dtype=torch.uint8, device=gu.DEV)
    sc = given(s, cks, "e4m3", saved, t["keep"], cl.ROWS_FULL)
    dout = gu.bf16(t["dout"])
    idx, cu, nk = gu.compact(t["keep"])
    run = lambda: cl.collider_layer_bwd_ckpt(L.desc, L.weights, sc, dout, cl.ROWS_FULL, idx, cu, nk, L.grads,  # noqa: E731
                                             cl.ROWS_FULL, ws)
    run()
    want = L.results()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for _ in range(2):
        L.dx.fill_(9)
        for v in L.grads_t.values():
            v.fill_(9)
        g.replay()
        got = L.results()
        for k in want:
            assert np.array_equal(got[k], want[k]), k
    nk.zero_()
    cu.zero_()
    g.replay()
    got = L.results()
    cl.collider_check()
    for k in got:
        assert np.all(got[k] == 0), k


def test_refusals():
    s, w, t, saved, cks = case("llama", "e4m3")
    L = gu.DeviceLayer(s, w, saved)
    ws = torch.empty(cl.collider_layer_ckpt_workspace_size(L.desc), dtype=torch.uint8, device=gu.DEV)
    idx, cu, nk = gu.compact(t["keep"])
    dout = gu.bf16(t["dout"])

    def refused(text, sc, i=idx, d=dout, wsp=ws):
        with pytest.raises(cl.ColliderError, match=text):
            cl.collider_layer_bwd_ckpt(L.desc, L.weights, sc, d, cl.ROWS_FULL, i, cu, nk, L.grads, cl.ROWS_FULL, wsp)
    ok = given(s, cks, "e4m3", saved, t["keep"], cl.ROWS_FULL)
    refused("index", ok, i=None)
    refused("workspace", ok, wsp=ws[:1024])
    ok.rows = 4
    refused("rows", ok)
    part = given(s, {k: v for k, v in cks.items() if k != "h"}, "e4m3", saved, t["keep"], cl.ROWS_FULL)
    refused("null checkpoint", part)
    host = given(s, cks, "e4m3", saved, t["keep"], cl.ROWS_FULL)
    c, e = host.buffers["up"].buffers
    host.up = cl.ckpt(cl.CKPT_E4M3, c.cpu(), e)
    refused("memory", host)
