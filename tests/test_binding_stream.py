"""The stream a call of the binding takes when none is given: torch's current one, by its raw handle where torch has the
function for that, else through the public API."""
import types

import torch

from sparse_backward_gemm_gb300 import collider


def test_given_streams():
    assert collider._stream(0) == 0 and collider._stream(7) == 7
    assert collider._stream(types.SimpleNamespace(cuda_stream=9)) == 9


def test_current_stream_by_its_raw_handle(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 100 + device, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    assert collider._stream(None) == 103


def test_current_stream_of_a_torch_without_it(monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=55))
    assert collider._stream(None) == 55
