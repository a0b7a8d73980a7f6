"""The compiled marshalling answers None to what is not the ordinary case, without touching a device (host tensors here)."""
import pytest
import torch

import gated_deltanet_gdr_b200 as gdr
from gated_deltanet_gdr_b200 import build as gbuild


@pytest.fixture(scope="module")
def m():
    gbuild.build()
    gdr.lib()
    assert gdr._quick is not None
    return gdr._quick


def test_host_tensors_and_other_objects_are_left_to_python(m):
    e, p, i = torch.zeros(1, 1, 4, 4), torch.zeros(3, 1, 4), torch.zeros(4, dtype=torch.int32)
    N, F, T = None, False, True
    assert m.scan_fwd(e, e, N, N, N, N, N, F, T, F, 0, 0) is None
    assert m.scan_fwd(3, "x", N, N, N, N, N, F, T, F, 0, 0) is None
    assert m.scan_bwd(e, e, e, e, N, N, N, N, N, F, T, 0, 0) is None
    assert m.scan_step(e, e, p, i, N, N, N, F, F, 0, 0) is None
    assert m.conv1d_bwd(p, p, e, e, e, *[N] * 9, 0, 0) is None
    for pools in (p, [p], (), [], 5, N):
        assert m.slot_copy(pools, i, i, 0, 0) is None
        assert m.slot_fork(pools, i, i, N, 0, 0) is None
        assert m.slot_compact(pools, i, N, N, 0, 0) is None
        assert m.slot_free(pools, i, N, 0, 0) is None


def test_wrong_numbers_of_arguments(m):
    for f in (m.scan_fwd, m.scan_bwd, m.scan_step, m.conv1d_bwd, m.slot_copy, m.slot_fork, m.slot_compact, m.slot_free, m.bind):
        with pytest.raises(TypeError):
            f(1)


def test_another_torch_is_marshalled_in_python(m, monkeypatch):
    L = gdr.lib()
    monkeypatch.setattr(gdr, "_quick", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    gdr._load_marshal(L)
    assert gdr._quick is None
    monkeypatch.undo()
    assert m.torch_version == torch.__version__ and gdr._quick is m
