"""Argument errors of the checkpoint and residual-join entry points: synchronous, before any CUDA call, so no GPU
is needed.  The addresses are never dereferenced."""
import pytest

import sparse_backward_gemm_gb300 as cl

FAKE = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def built():
    from sparse_backward_gemm_gb300 import build
    build.build()


def refused(status, text, fn, *a, **kw):
    with pytest.raises(cl.ColliderError) as e:
        fn(*a, stream=0, **kw)
    assert e.value.status == status and text in str(e.value), str(e.value)


def ck(**kw):
    return cl.Ckpt(**dict(dict(format=cl.CKPT_E4M3, code=FAKE, exps=FAKE + 1, code_ld=256, exp_ld=8), **kw))


BAD, NO = cl.ERR_INVALID_ARG, cl.ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,status,text", [
    (dict(format=2), NO, "format"), (dict(code=None), BAD, "null"), (dict(exps=None), BAD, "null"),
    (dict(code=FAKE + 8), BAD, "aligned"), (dict(code_ld=240), BAD, "codes"), (dict(code_ld=264), BAD, "codes"),
    (dict(exp_ld=7), BAD, "exponents"),
])
def test_checkpoints(kw, status, text):
    q = ck(**kw)
    refused(status, text, cl.collider_ckpt_pack, cl.BF16, FAKE, 256, 4, 256, None, None, q)
    refused(status, text, cl.collider_ckpt_unpack, cl.BF16, q, cl.ROWS_FULL, 4, 256, None, None, FAKE, 256, cl.ROWS_FULL)
    refused(status, text, cl.collider_linear_bwd_ckpt, 4, 256, 64, q, cl.ROWS_FULL, FAKE, FAKE, cl.ROWS_FULL, FAKE, FAKE,
            FAKE, cl.ROWS_FULL, FAKE, None, None)


@pytest.mark.parametrize("args,status,text", [
    ((7, FAKE, 256, 4, 256, None, None), NO, "dtype"), ((cl.BF16, None, 256, 4, 256, None, None), BAD, "null"),
    ((cl.BF16, FAKE, 256, 4, 256, FAKE, None), BAD, "only one"), ((cl.BF16, FAKE, 256, 0, 256, None, None), BAD, "M"),
    ((cl.BF16, FAKE, 256, (1 << 30) + 1, 256, None, None), BAD, "M"),
    ((cl.BF16, FAKE, 256, 4, 250, None, None), NO, "32"), ((cl.BF16, FAKE, 256, 4, 0, None, None), NO, "32"),
    ((cl.BF16, FAKE + 2, 256, 4, 256, None, None), BAD, "aligned"), ((cl.BF16, FAKE, 248, 4, 256, None, None), BAD, "stride"),
    ((cl.BF16, FAKE, 260, 4, 256, None, None), BAD, "stride"), ((cl.F32, FAKE, 258, 4, 256, None, None), BAD, "stride"),
])
def test_pack_arguments(args, status, text):
    refused(status, text, cl.collider_ckpt_pack, *args, ck())


def test_unpack_arguments():
    f = cl.collider_ckpt_unpack
    refused(BAD, "rows", f, cl.BF16, ck(), 2, 4, 256, None, None, FAKE, 256, cl.ROWS_FULL)
    refused(BAD, "rows", f, cl.BF16, ck(), cl.ROWS_FULL, 4, 256, None, None, FAKE, 256, 5)
    refused(BAD, "null", f, cl.BF16, ck(), cl.ROWS_FULL, 4, 256, None, None, None, 256, cl.ROWS_FULL)
    refused(BAD, "only one", f, cl.BF16, ck(), cl.ROWS_FULL, 4, 256, None, FAKE, FAKE, 256, cl.ROWS_FULL)
    refused(NO, "dtype", f, 3, ck(), cl.ROWS_FULL, 4, 256, None, None, FAKE, 256, cl.ROWS_FULL)


def test_linear_arguments():
    def lin(status, text, M=4, K=256, N=64, X=ck(), W=FAKE, dY=FAKE, idx=FAKE, nk=FAKE, dX=FAKE, dW=FAKE, db=None, rows=0):
        refused(status, text, cl.collider_linear_bwd_ckpt, M, K, N, X, rows, W, dY, cl.ROWS_FULL, idx, nk, dX,
                cl.ROWS_FULL, dW, db, None)
    lin(BAD, "sizes", M=0)
    lin(BAD, "null", dY=None)
    lin(BAD, "null", idx=None)
    lin(BAD, "dX needs W", W=None)
    lin(BAD, "rows", rows=3)
    lin(BAD, "misaligned", idx=FAKE + 2)
    lin(NO, "% 8", N=60)
    lin(BAD, "aligned", dX=FAKE + 4)
    lin(BAD, "null checkpoint", X=None)
    lin(BAD, "workspace")
    lin(BAD, "workspace", X=None, dW=None)            # without dW no checkpoint is needed
    assert cl.collider_linear_ckpt_workspace_size(8192, 2048, 5632) > 0


def test_linear_in_place_of_compact_rows():
    """A FULL dX gets its zeros while dY is still read: not over a COMPACT dY."""
    for dy_rows, dx_rows, text in ((cl.ROWS_COMPACT, cl.ROWS_FULL, "alias"), (cl.ROWS_FULL, cl.ROWS_FULL, "workspace"),
                                   (cl.ROWS_COMPACT, cl.ROWS_COMPACT, "workspace")):
        refused(BAD, text, cl.collider_linear_bwd_ckpt, 4, 256, 256, ck(), cl.ROWS_FULL, FAKE, 2 * FAKE, dy_rows, FAKE, FAKE,
                2 * FAKE, dx_rows, FAKE, None, None)


def layer(arch):
    d = cl.LayerDesc(B=1, T=64, D=256, H=4, Hkv=4, dh=64, F=256, rotary_dim=32, rope_base=1e4, eps=1e-5, arch=arch,
                     norm=cl.NORM_RMS if arch == cl.ARCH_LLAMA else cl.NORM_LAYER,
                     act=cl.ACT_SWIGLU if arch == cl.ARCH_LLAMA else cl.ACT_GELU_TANH)
    q = lambda n: ck(code_ld=n, exp_ld=n // 32)  # noqa: E731
    return d, dict(x=q(256), a=q(256), qkv=q(768), o=q(256), h=q(256), up=q(512), rstd1=FAKE, lse=FAKE, rstd2=FAKE, mean1=FAKE)


@pytest.mark.parametrize("arch", [cl.ARCH_LLAMA, cl.ARCH_PHI])
def test_layer_arguments(arch):
    d, saved = layer(arch)

    def run(status, text, dout_rows=cl.ROWS_FULL, dx_rows=cl.ROWS_FULL, idx=FAKE, **kw):
        sc = cl.LayerSavedCkpt(rows=cl.ROWS_FULL)
        for k, v in dict(saved, **kw).items():
            setattr(sc, k, v)
        refused(status, text, cl.collider_layer_bwd_ckpt, d, cl.LayerWeights(), sc, FAKE, dout_rows, idx, FAKE, FAKE,
                cl.LayerGrads(), dx_rows, None)
    run(BAD, "workspace")
    run(BAD, "rows", rows=2)
    run(BAD, "rows", dout_rows=2)
    run(BAD, "rows", dx_rows=-1)
    run(BAD, "null", idx=None)
    run(NO, "format", x=ck(format=3))
    run(BAD, "codes", qkv=ck())
    for k in ("mean1", "rstd1", "lse", "rstd2"):
        run(BAD, "misaligned", **{k: FAKE + 2})


def desc(**kw):
    return cl.ResidualNormDesc(**dict(dict(dtype=cl.BF16, B=2, T=8, D=64, norm=cl.NORM_RMS, post=1, pre=1, eps=1e-5,
                                           res_scale=1.0, gate_rows=1), **kw))


def par(**kw):
    return cl.ResidualNormParams(**dict(dict(post_w=FAKE, gate=FAKE, pre_w=FAKE), **kw))


DESC = [(dict(dtype=2), NO, "dtype"), (dict(norm=2), NO, "norm"), (dict(B=0), BAD, "B, T"),
        (dict(B=1 << 16, T=1 << 16), BAD, "2^30"), (dict(D=60), NO, "multiple of 8"), (dict(D=8200), NO, "8192"),
        (dict(D=0), NO, "D"), (dict(eps=0.0), BAD, "eps"), (dict(eps=float("nan")), BAD, "eps"),
        (dict(res_scale=float("inf")), BAD, "res_scale"), (dict(gate_rows=3), BAD, "gate_rows"),
        (dict(gate_rows=-1), BAD, "gate_rows"), (dict(x_ld=56), BAD, "stride"), (dict(a_ld=68), BAD, "stride"),
        (dict(y_ld=-64), BAD, "stride"), (dict(dtype=cl.F32, h_ld=66), BAD, "stride")]


@pytest.mark.parametrize("kw,status,text", DESC)
def test_join_desc(kw, status, text):
    d = desc(**kw)
    out = cl.ResidualNormOut(h=FAKE, a=2 * FAKE, rstd_y=FAKE, rstd_h=FAKE)
    refused(status, text, cl.collider_residual_norm_fwd, d, par(), 3 * FAKE, 4 * FAKE, out)
    sv = cl.ResidualNormSaved(y=FAKE, h=FAKE, rstd_y=FAKE, rstd_h=FAKE)
    g = cl.ResidualNormGrads(dx=5 * FAKE, dy=6 * FAKE)
    refused(status, text, cl.collider_residual_norm_bwd, d, par(), sv, cl.ROWS_FULL, FAKE, FAKE, cl.ROWS_FULL, None, None,
            None, g, cl.ROWS_FULL, None)
    assert cl.collider_residual_norm_bwd_workspace_size(d) == 0


def test_join_forward_arguments():
    def fwd(status, text, d=desc(), p=par(), x=3 * FAKE, y=4 * FAKE, **out):
        o = cl.ResidualNormOut(**dict(dict(h=FAKE, a=2 * FAKE, rstd_y=FAKE, rstd_h=FAKE), **out))
        refused(status, text, cl.collider_residual_norm_fwd, d, p, x, y, o)
    fwd(BAD, "null x", x=None)
    fwd(BAD, "null", p=par(post_w=None))
    fwd(BAD, "null", p=par(gate=None))
    fwd(BAD, "not ask", p=par(post_b=FAKE))                       # RMSNorm has no bias
    fwd(BAD, "not ask", d=desc(gate_rows=0))
    fwd(BAD, "not ask", d=desc(pre=0))
    fwd(BAD, "without y", y=None)                                 # post norm and gate without y
    fwd(BAD, "without y", d=desc(post=0, gate_rows=0, res_scale=2.0), p=par(post_w=None, gate=None), y=None)
    fwd(BAD, "without y", d=desc(post=0, pre=0, gate_rows=0), p=par(post_w=None, gate=None, pre_w=None), y=None)
    fwd(BAD, "h is written", h=None)
    fwd(BAD, "h is written", d=desc(post=0, gate_rows=0), p=par(post_w=None, gate=None), y=None)
    fwd(BAD, "rstd_h", a=None)
    fwd(BAD, "rstd_h", rstd_h=None)
    fwd(BAD, "mean_h", d=desc(norm=cl.NORM_LAYER))
    fwd(BAD, "rstd_y", rstd_y=None)
    fwd(BAD, "alias", a=3 * FAKE)
    fwd(BAD, "stride", d=desc(h_ld=128), h=3 * FAKE)              # in place with another stride
    fwd(BAD, "aligned", x=3 * FAKE + 2)
    fwd(BAD, "aligned", p=par(res_w=FAKE + 4))
    fwd(BAD, "4-byte", rstd_h=FAKE + 2)
    fwd(BAD, "stride", d=desc(x_ld=(1 << 28) + 8))


def test_join_backward_arguments():
    def bwd(status, text, d=desc(), p=par(), da=7 * FAKE, dh=8 * FAKE, idx=(None, None, None), rows=(0, 0, 0), sv=None, **g):
        s = cl.residual_norm_saved(**dict(dict(y=FAKE, h=2 * FAKE, rstd_y=FAKE, rstd_h=FAKE), **(sv or {})))
        gr = cl.ResidualNormGrads(**dict(dict(dx=5 * FAKE, dy=6 * FAKE), **g))
        refused(status, text, cl.collider_residual_norm_bwd, d, p, s, rows[0], da, dh, rows[1], *idx, gr, rows[2], None)
    bwd(BAD, "workspace")
    bwd(BAD, "only some", idx=(FAKE, None, FAKE))
    bwd(BAD, "only some", idx=(FAKE, FAKE, None))
    bwd(BAD, "rows", rows=(0, 2, 0))
    bwd(BAD, "needs da", da=None)
    bwd(BAD, "needs da", sv=dict(h=None))
    bwd(BAD, "needs da", d=desc(norm=cl.NORM_LAYER))              # LayerNorm: the means too
    bwd(BAD, "rstd_y", sv=dict(rstd_y=None))
    bwd(BAD, "dh is needed", d=desc(pre=0), p=par(pre_w=None), da=None, dh=None)
    bwd(BAD, "dres_w needs x", p=par(res_w=FAKE), dres_w=FAKE)
    bwd(BAD, "dy with y", dy=None)
    bwd(BAD, "dx is written", dx=None)
    bwd(BAD, "not both", sv=dict(y_ckpt=ck()))
    bwd(NO, "same form", sv=dict(h=None, h_ckpt=ck()))
    bwd(NO, "same form", sv=dict(h=None, h_ckpt=ck(), y=None, y_ckpt=ck(format=cl.CKPT_INT8)))
    bwd(NO, "32", d=desc(D=72), sv=dict(h=None, h_ckpt=ck(), y=None, y_ckpt=ck()))
    bwd(BAD, "4-byte", sv=dict(rstd_y=FAKE + 1))
    bwd(BAD, "4-byte", dgate=FAKE + 3)
    bwd(BAD, "4-byte", idx=(FAKE + 2, FAKE, FAKE))
    bwd(BAD, "alias", dx=7 * FAKE)
    bwd(BAD, "alias", dy=8 * FAKE)
    bwd(BAD, "alias", dx=8 * FAKE, rows=(0, 1, 0))                # in place needs the same rows
    bwd(BAD, "workspace", dx=8 * FAKE)
    first = dict(p=par(post_w=None, gate=None), sv=dict(y=None, rstd_y=None), dy=None)   # without y, x stands for h
    bwd(BAD, "workspace", d=desc(post=0, gate_rows=0, x_ld=128, h_ld=128), **first)
    bwd(BAD, "row stride", d=desc(post=0, gate_rows=0, x_ld=128), **first)


def test_binding_helpers():
    import torch
    with pytest.raises(TypeError):
        cl.residual_norm_grads(dz=None)
    with pytest.raises(TypeError):
        cl.ckpt(cl.CKPT_E4M3, torch.zeros(4, 64, dtype=torch.uint8).t(), torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(TypeError):
        cl.ckpt(cl.CKPT_E4M3, torch.zeros(4, 64), torch.zeros(4, 2, dtype=torch.uint8))
    q = cl.ckpt(cl.CKPT_INT8, torch.zeros(4, 80, dtype=torch.uint8)[:, :64], torch.zeros(4, 2, dtype=torch.uint8))
    assert (q.code_ld, q.exp_ld, q.format) == (80, 2, cl.CKPT_INT8)
    d = desc()
    small, big = (cl.collider_residual_norm_bwd_workspace_size(desc(B=8, T=2048, D=2048, gate_rows=g)) for g in (1, 8))
    assert 0 < cl.collider_residual_norm_bwd_workspace_size(d) < small < big
