"""A gradient of a parameter that the residual join does not have is refused, rather than left as it was.  Host checks
alone; the addresses are never dereferenced."""
import pytest

import sparse_backward_gemm_gb300 as cl

FAKE = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def built():
    from sparse_backward_gemm_gb300 import build
    build.build()


def error(norm=cl.NORM_RMS, post=1, pre=1, gate_rows=1, res=True, branch=True, **g):
    d = cl.ResidualNormDesc(dtype=cl.BF16, B=2, T=8, D=64, norm=norm, post=post, pre=pre, eps=1e-5, res_scale=1.0,
                            gate_rows=gate_rows)
    p = cl.ResidualNormParams(post_w=FAKE if post else None, pre_w=FAKE if pre else None, gate=FAKE if gate_rows else None,
                              res_w=FAKE if res else None)
    sv = cl.residual_norm_saved(y=2 * FAKE if branch else None, h=3 * FAKE, x=4 * FAKE, rstd_y=FAKE, rstd_h=FAKE, mean_y=FAKE,
                                mean_h=FAKE)
    gr = cl.ResidualNormGrads(dx=5 * FAKE, dy=6 * FAKE if branch else None, **g)
    with pytest.raises(cl.ColliderError) as e:
        cl.collider_residual_norm_bwd(d, p, sv, cl.ROWS_FULL, 7 * FAKE if pre else None, 8 * FAKE, cl.ROWS_FULL, None, None,
                                      None, gr, cl.ROWS_FULL, None, stream=0)
    assert e.value.status == cl.ERR_INVALID_ARG
    return str(e.value)


@pytest.mark.parametrize("kw", [
    dict(post=0, dpost_w=FAKE), dict(pre=0, dpre_w=FAKE), dict(gate_rows=0, dgate=FAKE), dict(res=False, dres_w=FAKE),
    dict(dpost_b=FAKE), dict(dpre_b=FAKE),                                      # RMSNorm has no bias
    dict(norm=cl.NORM_LAYER, post=0, dpost_b=FAKE), dict(norm=cl.NORM_LAYER, pre=0, dpre_b=FAKE),
    dict(branch=False, post=0, gate_rows=0, res=False, dgate=FAKE), dict(branch=False, post=0, gate_rows=0, res=False, dres_w=FAKE),
])
def test_refused(kw):
    assert "does not ask for" in error(**kw)


@pytest.mark.parametrize("kw", [
    dict(), dict(dpost_w=FAKE, dpre_w=FAKE, dgate=FAKE, dres_w=FAKE),
    dict(norm=cl.NORM_LAYER, dpost_b=FAKE, dpre_b=FAKE),                        # biases that are 0 for want of a vector
    dict(branch=False, post=0, gate_rows=0, res=False, dpre_w=FAKE),
])
def test_asked_for(kw):
    assert "workspace" in error(**kw)
