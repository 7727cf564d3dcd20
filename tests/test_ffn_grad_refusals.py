"""Argument errors of the feed-forward and gradient-norm entry points: synchronous, before any CUDA call, so no GPU is
needed.  The addresses are never dereferenced."""
import math

import pytest

import sparse_backward_gemm_gb300 as cl

MB = 1 << 20
BAD, NO = cl.ERR_INVALID_ARG, cl.ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def built():
    from sparse_backward_gemm_gb300 import build
    build.build()


def refused(status, text, fn, *a):
    with pytest.raises(cl.ColliderError) as e:
        fn(*a, stream=0)
    assert e.value.status == status and text in str(e.value), str(e.value)


def desc(**kw):
    return cl.FfnDesc(**dict(dict(M=64, D=64, F=128, act=cl.GLU_SILU, grad_dtype=cl.BF16), **kw))


DESCS = [(dict(act=2), NO, "act"), (dict(grad_dtype=5), NO, "grad_dtype"), (dict(M=0), BAD, "M"), (dict(M=-1), BAD, "M"),
         (dict(M=(1 << 30) + 1), BAD, "M"), (dict(D=60), NO, "multiples of 8"), (dict(F=4), NO, "multiples of 8"),
         (dict(F=0), NO, "multiples of 8"), (dict(D=(1 << 20) + 8), NO, "2^20"), (dict(x_ld=-8), BAD, "negative"),
         (dict(x_ld=56), BAD, "strides"), (dict(x_ld=68), BAD, "strides"), (dict(up_ld=248), BAD, "strides"),
         (dict(y_ld=72 + 4), BAD, "strides"), (dict(y_ld=(1 << 28) + 8), BAD, "strides")]


@pytest.mark.parametrize("kw,status,text", DESCS)
def test_descs(kw, status, text):
    d = desc(**kw)
    refused(status, text, cl.collider_ffn_fwd, d, MB, 2 * MB, 3 * MB, None, 4 * MB, None)
    refused(status, text, cl.collider_ffn_bwd, d, MB, 2 * MB, 3 * MB, 4 * MB, 0, 5 * MB, 0, None, None, 6 * MB, 0, 7 * MB, 8 * MB, None)
    assert cl.collider_ffn_fwd_workspace_size(d) == 0 and cl.collider_ffn_bwd_workspace_size(d) == 0


@pytest.mark.parametrize("kw,text", [
    (dict(x=None), "null"), (dict(w_up=None), "null"), (dict(w_down=None), "null"), (dict(y=None), "null"),
    (dict(x=MB + 8), "aligned"), (dict(up=5 * MB + 2), "aligned"), (dict(y=MB), "alias"), (dict(y=MB + 64 * 128 - 16), "alias"),
    (dict(up=4 * MB), "alias"), (dict(up=2 * MB + 64 * 512 - 16), "alias"), (dict(y=3 * MB), "alias"),
    (dict(), "workspace"), (dict(y=MB + 64 * 128), "workspace"),
])
def test_forward_arguments(kw, text):
    a = dict(dict(x=MB, w_up=2 * MB, w_down=3 * MB, up=5 * MB, y=4 * MB), **kw)
    refused(BAD, text, cl.collider_ffn_fwd, desc(), a["x"], a["w_up"], a["w_down"], a["up"], a["y"], None)


@pytest.mark.parametrize("kw,text", [
    (dict(w_down=None), "null"), (dict(up=None), "null"), (dict(dy=None), "null"), (dict(w_up=None), "dx needs"),
    (dict(x=None), "dw_up needs"), (dict(saved_rows=2), "rows"), (dict(dy_rows=-1), "rows"), (dict(dx_rows=7), "rows"),
    (dict(idx=9 * MB), "only one"), (dict(nk=9 * MB), "only one"), (dict(idx=9 * MB + 2, nk=10 * MB), "misaligned"),
    (dict(dx=6 * MB + 8), "aligned"), (dict(dw_up=7 * MB + 4), "aligned"), (dict(dx=3 * MB), "alias"),
    (dict(dx=5 * MB), "alias"), (dict(dx=4 * MB + 64 * 512 - 16), "alias"), (dict(dw_up=MB), "alias"),
    (dict(dw_up=8 * MB - 16), "alias"), (dict(dw_down=2 * MB), "alias"), (dict(idx=7 * MB, nk=10 * MB), "alias"),
    (dict(), "workspace"), (dict(dx=None, w_up=None), "workspace"), (dict(dw_up=None, x=None), "workspace"),
])
def test_backward_arguments(kw, text):
    a = dict(dict(w_up=MB, w_down=2 * MB, x=3 * MB, up=4 * MB, saved_rows=0, dy=5 * MB, dy_rows=0, idx=None, nk=None,
                  dx=6 * MB, dx_rows=0, dw_up=7 * MB, dw_down=8 * MB), **kw)
    refused(BAD, text, cl.collider_ffn_bwd, desc(), *a.values(), None)


def test_compact_rows_alias_by_their_first():
    """Of COMPACT rows the host knows the first alone."""
    common = dict(w_up=MB, w_down=2 * MB, x=3 * MB, up=4 * MB)
    for dx, text in ((5 * MB, "alias"), (5 * MB + 112, "alias"), (5 * MB + 128, "workspace")):
        refused(BAD, text, cl.collider_ffn_bwd, desc(), *common.values(), 1, 5 * MB, 1, 9 * MB, 10 * MB, dx, 1, None, None, None)


def grads(*items):
    return (cl.Grad * max(1, len(items)))(*[cl.Grad(*i) for i in items])


@pytest.mark.parametrize("items,count,kw,status,text", [
    ([(MB, 8, 0)], -1, {}, BAD, "count"), ([(MB, 8, 0)], (1 << 20) + 1, {}, BAD, "count"), ([(MB, 8, 2)], 1, {}, NO, "dtype"),
    ([(MB, -1, 0)], 1, {}, BAD, "size"), ([(None, 8, 0)], 1, {}, BAD, "null"), ([(MB + 2, 8, 0)], 1, {}, BAD, "aligned"),
    ([(MB + 1, 8, 1)], 1, {}, BAD, "aligned"), ([(MB, 1 << 40, 0), (1 << 50, 1, 0)], 2, {}, BAD, "2^40"),
    ([(MB, 8, 0)], 1, dict(kind=2), NO, "kind"), ([(MB, 8, 0)], 1, dict(scale=0.0), BAD, "scale"),
    ([(MB, 8, 0)], 1, dict(scale=-1.0), BAD, "scale"), ([(MB, 8, 0)], 1, dict(scale=math.inf), BAD, "scale"),
    ([(MB, 8, 0)], 1, dict(scale=math.nan), BAD, "scale"), ([(MB, 8, 0)], 1, dict(norm=2 * MB + 1), BAD, "aligned"),
    ([(MB, 8, 0)], 1, dict(norm=3 * MB), BAD, "alias"), ([(2 * MB - 28, 8, 0)], 1, {}, BAD, "lies in gradient 0"),
    ([(MB, 8, 0), (MB + 32, 8, 0)], 2, {}, BAD, "workspace"), ([(MB, 8, 0), (None, 0, 1)], 2, {}, BAD, "workspace"),
    ([], 0, {}, BAD, "workspace"),
])
def test_gradient_lists(items, count, kw, status, text):
    a = dict(dict(kind=cl.GRAD_NORM_L2, scale=1.0, norm=2 * MB, norms=3 * MB), **kw)
    g = grads(*items)
    refused(status, text, cl.collider_grad_norm, g, count, a["kind"], a["scale"], a["norm"], a["norms"], None)
    refused(status, text, cl.collider_grad_clip, g, count, a["kind"], a["scale"], 1.0, a["norm"], a["norms"], 4 * MB, None)


def test_clipping_refuses_shared_values():
    shared = grads((MB + 32, 8, 0), (4 * MB, 8, 1), (MB, 9, 0))
    refused(BAD, "overlap", cl.collider_grad_clip, shared, 3, 0, 1.0, 1.0, 2 * MB, None, None, None)
    refused(BAD, "overlap", cl.collider_grad_clip, grads((MB, 8, 0), (MB, 8, 0)), 2, 0, 1.0, 1.0, None, None, None, None)
    refused(BAD, "workspace", cl.collider_grad_norm, shared, 3, 0, 1.0, 2 * MB, None, None)   # the norm alone takes it
    refused(BAD, "workspace", cl.collider_grad_clip, grads((MB + 32, 8, 0), (MB, 8, 0)), 2, 0, 1.0, 1.0, None, None, None, None)
    for m in (-1.0, math.nan):
        refused(BAD, "max_norm", cl.collider_grad_clip, grads((MB, 8, 0)), 1, 0, 1.0, m, None, None, None, None)
    refused(BAD, "workspace", cl.collider_grad_clip, grads((MB, 8, 0)), 1, 0, 1.0, math.inf, None, None, None, None)


def test_sizes():
    d = desc(M=8192, D=2048, F=5632)
    assert cl.collider_ffn_fwd_workspace_size(d) >= 8192 * 5632 * 2
    assert cl.collider_ffn_bwd_workspace_size(d) >= 8192 * (3 * 5632 + 2 * 2048) * 2
    assert cl.collider_grad_norm_workspace_size(None, 0) > 0 and cl.collider_grad_norm_workspace_size(None, -1) == 0


def test_grad_list_takes_contiguous_floats():
    import torch
    with pytest.raises(TypeError):
        cl.grad_list([torch.zeros(4, 4).T[:, :2]])
    with pytest.raises(TypeError):
        cl.grad_list([torch.zeros(4, dtype=torch.float64)])
    a = cl.grad_list([torch.zeros(3, 5), torch.zeros(0, dtype=torch.bfloat16)])
    assert [(g.n, g.dtype) for g in a] == [(15, cl.F32), (0, cl.BF16)]
