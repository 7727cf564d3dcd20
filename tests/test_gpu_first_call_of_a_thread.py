"""A host thread's first CUDA call may be one of the library's whose first step makes a tensor map."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

gu = pytest.importorskip("gpu_util")
cl = gu.cl


def test_attention_backward_first_in_a_thread():
    T, H, dh = 256, 4, 64
    gen = torch.Generator(device=gu.DEV).manual_seed(3)
    q, k, v, do = (torch.randn(T, H, dh, generator=gen, device=gu.DEV).bfloat16() for _ in range(4))
    lse = torch.logsumexp((torch.einsum("ihd,jhd->hij", q.float(), k.float()) / 8).tril(), -1).reshape(1, H, T).contiguous()
    import numpy as np
    idx, cu, nk = gu.compact(np.ones((1, T), bool))
    ws = torch.empty(cl.collider_attn_workspace_size(1, T, H, H, dh), dtype=torch.uint8, device=gu.DEV)
    out = [[torch.empty_like(q) for _ in range(3)] for _ in range(2)]

    def call(o):
        cl.collider_attn_bwd(1, T, H, H, dh, 1, 0.125, 0, 10000.0, q, k, v, None, do, H * dh, H * dh, H * dh, cl.ROWS_FULL, lse,
                             idx, cu, nk, *o, cl.ROWS_FULL, ws, stream=0)
        cl.collider_check(0)
    call(out[0])
    torch.cuda.synchronize()
    failed = []

    def work():
        try:
            call(out[1])
        except cl.ColliderError as e:
            failed.append(e)
    th = threading.Thread(target=work)
    th.start()
    th.join()
    torch.cuda.synchronize()
    assert not failed and all(torch.equal(a, b) for a, b in zip(*out))
