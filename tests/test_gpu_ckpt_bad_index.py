"""Unpacking 8-bit checkpoints with a kept index outside the rows."""
import numpy as np
import pytest
import torch

from oracle import ckpt as ock
import workloads

pytestmark = pytest.mark.gpu

gu = pytest.importorskip("gpu_util")
cl = gu.cl
FMT = {"e4m3": cl.CKPT_E4M3, "int8": cl.CKPT_INT8}
DT = {"bf16": (cl.BF16, torch.bfloat16), "f32": (cl.F32, torch.float32)}


def packed(v, fmt, dtype):
    M, N = v.shape
    cdt, tdt = DT[dtype]
    src = torch.from_numpy(v.astype(np.float32)).to(gu.DEV).to(tdt)
    q = cl.ckpt(FMT[fmt], torch.empty(M, N, dtype=torch.uint8, device=gu.DEV),
                torch.empty(M, N // 32, dtype=torch.uint8, device=gu.DEV))
    cl.collider_ckpt_pack(cdt, src, N, M, N, None, None, q)
    return src, q


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_unpack_with_an_index_outside_the_rows(fmt, dtype):
    """Reported; its row of a COMPACT output is zeros, and of a FULL one there is none.  The other rows are there."""
    M, N = 300, 96
    v = np.random.default_rng(5).normal(size=(M, N)).astype(np.float32).astype(np.float64)
    v = workloads.bf16_representable(v).astype(np.float64) if dtype == "bf16" else v
    cdt, tdt = DT[dtype]
    _, q = packed(v, fmt, dtype)
    val = ock.unpack(*ock.pack(v, fmt), fmt)
    kept = np.arange(0, M, 2)
    idx = np.full(M, -1)
    idx[: kept.size] = kept
    idx[kept.size - 1] = M + 9
    idx_t, nk = gu.i32(idx), gu.i32([kept.size])
    for rows in (cl.ROWS_COMPACT, cl.ROWS_FULL):
        dst = torch.full((M, N), 7.0, dtype=tdt, device=gu.DEV)
        cl.collider_ckpt_unpack(cdt, q, cl.ROWS_FULL, M, N, idx_t, nk, dst, N, rows)
        with pytest.raises(cl.ColliderError) as e:
            cl.collider_check()
        assert e.value.status == cl.ERR_INVALID_ARG
        got = gu.host(dst)
        if rows == cl.ROWS_COMPACT:
            assert np.array_equal(got[: kept.size - 1], val[kept[:-1]])
            assert np.all(got[kept.size - 1: 256] == 0) and np.all(got[256:] == 7)
        else:
            assert np.array_equal(got[kept[:-1]], val[kept[:-1]])
    # COMPACT rows of a checkpoint are not looked up: every row decodes
    dst = torch.full((M, N), 7.0, dtype=tdt, device=gu.DEV)
    cl.collider_ckpt_unpack(cdt, q, cl.ROWS_COMPACT, M, N, idx_t, nk, dst, N, cl.ROWS_COMPACT)
    cl.collider_check()
    assert np.array_equal(gu.host(dst)[: kept.size], val[: kept.size])
