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


BIG = 2 ** 32 + 5  # 5 in 32 bits


def meta(*shape, dtype=torch.uint8):
    return torch.empty(shape, dtype=dtype, device="meta")


class Anywhere:
    """a call whose tensors are not looked at"""
    dev, other, stream = 0, None, 0

    def ptr(self, t, name, dtype, shape):
        return 1 << 30


def test_sizes_past_32_bits_are_refused(monkeypatch):
    """The C entries take sizes as int: a larger one must not arrive as what its low 32 bits say."""
    monkeypatch.setattr(gdr, "_quick", None)  # (the compiled marshalling asks for the current device)
    monkeypatch.setattr(gdr, "_ready", lambda: None)
    c = Anywhere()
    with pytest.raises(ValueError, match="2\\^31"):
        gdr._pools(c, meta(BIG, 1))
    with pytest.raises(ValueError, match="2\\^31"):
        gdr._pools(c, [meta(BIG, 2), meta(BIG, 1)])
    with pytest.raises(ValueError, match="2\\^31"):
        gdr._list_i32(c, meta(BIG, dtype=torch.int32), "src")
    for shape in ((BIG, 1, 0, 1), (1, BIG, 0, 1), (0, 1, BIG, 1), (1, 1, 0, BIG)):
        with pytest.raises(ValueError, match="2\\^31"):
            gdr._sizes(meta(*shape, dtype=torch.float32), "x")
    with pytest.raises(ValueError, match="2\\^31"):
        gdr._scan_step_args(meta(1, 1, 1, 4, dtype=torch.float32), meta(1, 1, 1, 4, dtype=torch.float32),
                            meta(BIG, 1, 4, dtype=torch.float32), meta(1, dtype=torch.int32), None, None, False, None, False, None)
    e = meta(0, 1, BIG, 16, dtype=torch.float32)
    with pytest.raises(ValueError, match="2\\^31"):
        gdr.conv1d_bwd(meta(0, BIG, 48, dtype=torch.float32), meta(48, 4, dtype=torch.float32), e, e, e)
    assert gdr._pools(c, meta(2 ** 31 - 1, 1))[2] == 2 ** 31 - 1 and gdr._sizes(meta(1, 2, 3, 4), "x") == (1, 2, 3, 4)
