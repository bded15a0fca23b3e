"""The stream that a call of the binding runs on when none is given."""
import types

import pytest
import torch

import sparse_mixture_experts_router_gb300 as moe


@pytest.mark.parametrize("missing", ["_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_a_torch_without_the_handle_alone(monkeypatch, missing):
    monkeypatch.delattr(torch._C, missing, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=0x1230))
    monkeypatch.setattr(moe, "_current_stream", None)
    assert moe._stream(None) == 0x1230
    assert moe._stream(5) == 5 and moe._stream(types.SimpleNamespace(cuda_stream=7)) == 7


@pytest.mark.gpu
def test_the_current_stream():
    other = torch.cuda.Stream()
    assert moe._stream(None) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(other):
        assert moe._stream(None) == other.cuda_stream == moe._stream(other)
