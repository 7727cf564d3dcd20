"""8-bit checkpoints of the largest finite values on the GPU."""
import numpy as np
import pytest
import torch

from oracle import ckpt as ock
from test_oracle_ckpt_largest import largest
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
def test_largest_values(fmt, dtype):
    """Bit for bit the oracle, finite in f32 and in bf16."""
    v = largest()
    if dtype == "bf16":
        v = np.concatenate([v, -v])
        v = workloads.bf16_representable(np.clip(v, -(2.0 - 2.0 ** -7) * 2.0 ** 127, (2.0 - 2.0 ** -7) * 2.0 ** 127))
    v = np.concatenate([np.asarray(v, np.float64), np.asarray(v, np.float64)[:, ::-1]], axis=1)
    src, q = packed(v, fmt, dtype)
    code, exps = ock.pack(v, fmt)
    assert np.array_equal(q.buffers[0].cpu().numpy(), code) and np.array_equal(q.buffers[1].cpu().numpy(), exps)
    for cdt, tdt in DT.values():
        dst = torch.empty(v.shape, dtype=tdt, device=gu.DEV)
        cl.collider_ckpt_unpack(cdt, q, 0, *v.shape, None, None, dst, v.shape[1], 0)
        cl.collider_check()
        assert bool(torch.isfinite(dst).all())
        assert np.array_equal(gu.host(dst), ock.unpack(code, exps, fmt))
