"""The residual join's backward takes y and h saved in one form: every mixture of rows and checkpoints is refused,
whichever of the two is the checkpoint.  Host checks alone; the addresses are never dereferenced."""
import pytest

import sparse_backward_gemm_gb300 as cl

FAKE = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def built():
    from sparse_backward_gemm_gb300 import build
    build.build()


def ck(fmt, at):
    return cl.Ckpt(format=fmt, code=at, exps=at + FAKE // 2, code_ld=64, exp_ld=2)


FORMS = {"rows": None, "e4m3": cl.CKPT_E4M3, "int8": cl.CKPT_INT8}


@pytest.mark.parametrize("norm", [cl.NORM_RMS, cl.NORM_LAYER])
@pytest.mark.parametrize("post", [0, 1])
@pytest.mark.parametrize("y", list(FORMS))
@pytest.mark.parametrize("h", list(FORMS))
def test_y_and_h_are_saved_in_one_form(y, h, post, norm):
    d = cl.ResidualNormDesc(dtype=cl.BF16, B=2, T=8, D=64, norm=norm, post=post, pre=1, eps=1e-5, res_scale=1.0)
    p = cl.ResidualNormParams(post_w=FAKE if post else None, pre_w=FAKE)
    sv = dict(rstd_y=FAKE, rstd_h=FAKE, mean_y=FAKE, mean_h=FAKE)
    for k, form, at in (("y", y, 2 * FAKE), ("h", h, 3 * FAKE)):
        sv[k if form == "rows" else k + "_ckpt"] = at if form == "rows" else ck(FORMS[form], at)
    g = cl.ResidualNormGrads(dx=5 * FAKE, dy=6 * FAKE)
    with pytest.raises(cl.ColliderError) as e:
        cl.collider_residual_norm_bwd(d, p, cl.residual_norm_saved(**sv), cl.ROWS_FULL, 7 * FAKE, 8 * FAKE, cl.ROWS_FULL,
                                      None, None, None, g, cl.ROWS_FULL, None, stream=0)
    # (a call that is right but for its missing workspace is refused for that)
    status, text = (cl.ERR_INVALID_ARG, "workspace") if y == h else (cl.ERR_UNSUPPORTED, "same form")
    assert e.value.status == status and text in str(e.value), str(e.value)
