"""The binding's gradient calls look no further than the list they are given (the C side trusts the count)."""
import pytest

import sparse_backward_gemm_gb300 as cl

MB = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def built():
    from sparse_backward_gemm_gb300 import build
    build.build()


@pytest.mark.parametrize("count,size", [(2, 1), (1, 0), (200, 3), (1 << 20, 5)])
def test_a_count_beyond_the_list(count, size):
    g = (cl.Grad * size)(*[cl.Grad(MB + 64 * i, 8, cl.F32) for i in range(size)])
    for call in (lambda: cl.collider_grad_norm(g, count, cl.GRAD_NORM_L2, 1.0, 2 * MB, None, None, stream=0),
                 lambda: cl.collider_grad_clip(g, count, cl.GRAD_NORM_L2, 1.0, 1.0, 2 * MB, None, None, None, stream=0)):
        with pytest.raises(cl.ColliderError) as e:
            call()
        assert e.value.status == cl.ERR_INVALID_ARG and f"a list of {size}" in str(e.value), str(e.value)


def test_a_part_of_the_list():
    g = cl.Grad * 3
    with pytest.raises(cl.ColliderError) as e:   # (as far as the missing workspace)
        cl.collider_grad_norm(g(*[cl.Grad(MB + 64 * i, 8, cl.F32) for i in range(3)]), 2, cl.GRAD_NORM_L2, 1.0, 2 * MB, None,
                              None, stream=0)
    assert "workspace" in str(e.value)
