"""The binding's own checks, on the host: device and stream of a call (no device is touched)."""
from types import SimpleNamespace

import pytest
import torch

import gated_deltanet_gdr_b200 as gdr


@pytest.mark.parametrize("handle", [0, 64, 128])
def test_a_stream_of_another_device_is_refused(monkeypatch, handle):
    """The default streams of all devices have the handle 0: the device tells them apart."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(gdr, "_raw_stream", lambda dev: 0 if handle == 0 else 64)
    there = SimpleNamespace(cuda_stream=handle, device=torch.device("cuda", 1))
    with pytest.raises(RuntimeError, match="current device cuda:0"):
        gdr._Call(there)
    here = gdr._Call(SimpleNamespace(cuda_stream=handle, device=torch.device("cuda", 0)))
    assert here.stream == handle and (here.other is None) == (handle != 128)
