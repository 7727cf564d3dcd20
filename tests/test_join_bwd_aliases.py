"""The outputs of the residual join's backward lie apart from everything it reads but dh: a row of theirs may be
written before another block has read the saved row there.  Host checks alone; the addresses are never dereferenced."""
import pytest

import sparse_backward_gemm_gb300 as cl

FAKE = 1 << 20
Y, H, X, DA, DH, DX, DY, EXPS, WS = (FAKE * (16 + 4 * i) for i in range(9))


@pytest.fixture(scope="module", autouse=True)
def built():
    from sparse_backward_gemm_gb300 import build
    build.build()


def error(eight=False, branch=True, pre=1, res=False, dres=True, **g):
    ck = lambda at: cl.Ckpt(format=cl.CKPT_E4M3, code=at, exps=at + EXPS, code_ld=64, exp_ld=2)  # noqa: E731
    d = cl.ResidualNormDesc(dtype=cl.BF16, B=2, T=8, D=64, norm=cl.NORM_RMS, post=0, pre=pre, eps=1e-5, res_scale=1.0)
    p = cl.ResidualNormParams(pre_w=FAKE if pre else None, res_w=FAKE if res else None)
    sv = dict(rstd_h=FAKE, x=X)
    if branch:
        sv.update(y_ckpt=ck(Y)) if eight else sv.update(y=Y)
    sv.update(h_ckpt=ck(H)) if eight else sv.update(h=H)
    gr = dict(dx=DX, dy=DY if branch else None, dres_w=FAKE if res and dres else None, **{})
    gr.update(g)
    with pytest.raises(cl.ColliderError) as e:
        cl.collider_residual_norm_bwd(d, p, cl.residual_norm_saved(**sv), cl.ROWS_FULL, DA if pre else None, DH, cl.ROWS_FULL,
                                      None, None, None, cl.ResidualNormGrads(**gr), cl.ROWS_COMPACT, None, stream=0)
    assert e.value.status == cl.ERR_INVALID_ARG
    return "alias" if "alias" in str(e.value) else "workspace" if "workspace" in str(e.value) else str(e.value)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("out", ["dx", "dy"])
def test_outputs_over_saved_tensors(eight, out):
    assert error(eight=eight, **{out: Y}) == "alias"
    assert error(eight=eight, **{out: H}) == "alias"
    assert error(eight=eight, res=True, **{out: X}) == "alias"
    if eight:
        assert error(eight=True, **{out: Y + EXPS}) == "alias" and error(eight=True, **{out: H + EXPS}) == "alias"


def test_first_norm_over_its_input():
    assert error(branch=False, dx=H) == "alias"


def test_calls_that_read_nothing_there():
    assert error() == "workspace" and error(eight=True, res=True) == "workspace"
    assert error(dx=X) == "workspace" and error(dx=X, res=True, dres=False) == "workspace"    # x is read for dres_w alone
    assert error(pre=0, dx=H) == "workspace"                                                  # h is read by the pre norm alone
