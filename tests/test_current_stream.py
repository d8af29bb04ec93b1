"""The binding's default stream (CPU only, on a torch whose CUDA calls are stood in for)."""
import types

import pytest
import torch

import bwd_qwen3_layer_gb300 as K


@pytest.mark.parametrize("has_raw", [True, False])
def test_calls_go_to_the_current_stream(monkeypatch, has_raw):
    """With torch's function for the bare handle, and on a torch that lacks it."""
    now = dict(device=1, streams={0: 0x100, 1: 0x200})
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now["device"])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=now["streams"][now["device"]]))
    if has_raw:
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: now["streams"][d], raising=False)
    else:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(K, "_current_stream", None)
    assert K._stream(None) == 0x200
    now["device"] = 0
    assert K._stream(None) == 0x100
    now["streams"][0] = 0x300                      # asked for at every call
    assert K._stream(None) == 0x300
    assert K._stream(0x55) == 0x55 and K._stream(types.SimpleNamespace(cuda_stream=0x66)) == 0x66
