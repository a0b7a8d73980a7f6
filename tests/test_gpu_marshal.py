"""The two ways a short call is marshalled (csrc/marshal.cpp, and Python for everything out of the ordinary) make the same
calls: equal results, outputs given or new, and the same refusals."""
import numpy as np
import pytest
import torch

import gated_deltanet_gdr_b200 as gdr
from tests._helpers import dev_i32

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["compiled", "python"])
def way(request, monkeypatch):
    gdr.lib()
    assert gdr._quick is not None, "the compiled marshalling is not built"
    if request.param == "python":
        monkeypatch.setattr(gdr, "_quick", None)
    return request.param


def calls():
    """every call in turn on the same inputs, returning what it returns"""
    torch.manual_seed(3)
    r = lambda *s: torch.randn(*s, device="cuda")
    x, g, s0 = r(2, 3, 70, 24).bfloat16(), -torch.rand(2, 3, 70, 24, device="cuda"), r(2, 3, 24)
    lens = dev_i32([70, 33])
    res = [gdr.scan_fwd(x, g), gdr.scan_fwd(x, g, s0, lens, mix=True, output_checkpoints=True, checkpoints=torch.zeros(2, 3, 2, 24, device="cuda")),
           gdr.scan_fwd(x, g, s0, output_final_state=False)]
    o, f, ck = gdr.scan_fwd(x, g, s0, output_checkpoints=True)
    mine = torch.empty_like(x), torch.empty_like(s0), torch.empty_like(ck)
    out = gdr.scan_fwd(x, g, s0, out=mine[0], final_state=mine[1], checkpoints=mine[2])
    assert all(u is v for u, v in zip(out, mine))
    res += [out, gdr.scan_bwd(x, g, ck, x), gdr.scan_bwd(x, g, ck, x, s0, lens, output_dinitial_state=False)]
    d = torch.empty_like(x), torch.empty_like(g), torch.empty_like(s0)
    out = gdr.scan_bwd(x, g, ck, x, s0, dx=d[0], dg=d[1], dinitial_state=d[2])
    assert all(u is v for u, v in zip(out, d))
    res.append(out)
    pool, idx = r(6, 3, 24), dev_i32([5, 1, 0, 2])
    x2, g2 = x[:, :, :2].contiguous(), g[:, :, :2].contiguous()
    for kw in ({}, {"per_token": True, "mix": True}):
        out, p = gdr.scan_step(x2, g2, pool, idx, dev_i32([2, 1]), dev_i32([1, 2]), **kw)
        assert p is pool
        res.append((out, p.clone()))
    mine = torch.empty_like(x2)
    assert gdr.scan_step(x2, g2, pool, idx.reshape(2, 2), out=mine)[0] is mine
    res.append((mine,))
    xc, w, b, st = r(2, 40, 96), r(96, 4), r(96), r(2, 96, 4)
    dq, dk, dv = r(2, 1, 40, 32), r(2, 1, 40, 32), r(2, 1, 40, 32)
    ws = torch.empty(gdr.conv1d_bwd_workspace_bytes(2, 40, 1, 1, 32, 32, 4) + 64, dtype=torch.uint8, device="cuda")
    res += [gdr.conv1d_bwd(xc, w, dq, dk, dv), gdr.conv1d_bwd(xc, w, dq, dk, dv, b, st, dev_i32([40, 7]), st, workspace=ws)]
    mine = [torch.empty_like(t) for t in res[-1]]
    out = gdr.conv1d_bwd(xc, w, dq, dk, dv, b, st, None, st, dx=mine[0], dweight=mine[1], dbias=mine[2], dconv_state=mine[3])
    assert all(u is v for u, v in zip(out, mine))
    res.append(out)
    pools = [r(8, 5), r(8, 3, 3).half(), torch.arange(8, device="cuda")]
    assert gdr.slot_copy(pools, dev_i32([1, 1]), dev_i32([2, 7])) is pools
    res.append([p.clone() for p in pools])
    one = pools[0]
    assert gdr.slot_copy(one, dev_i32([0]), dev_i32([3])) is one
    new = torch.empty(3, dtype=torch.int32, device="cuda")
    assert gdr.slot_fork(tuple(pools), dev_i32([6, 0, 4]), dev_i32([1, 1, 2]), new_slot_table=new) is new
    res.append([gdr.slot_fork(pools, dev_i32([6, 0, 4]), dev_i32([1, 1, 2])), new] + [p.clone() for p in pools])
    live = dev_i32([0, 1, 0, 0, 1, 0, 1, 0])
    a, n = torch.empty_like(live), torch.empty(1, dtype=torch.int32, device="cuda")
    out = gdr.slot_compact(pools, live, new_slot=a, n_live=n)
    assert out[0] is a and out[1] is n
    res.append(list(out) + list(gdr.slot_compact(pools, live)) + [p.clone() for p in pools])
    assert gdr.slot_free(pools, dev_i32([3, -1]), live) is pools
    gdr.slot_free(pools[1], dev_i32([4]))
    res.append([live] + [p.clone() for p in pools])
    assert gdr.get_error() == 0
    return res


def test_both_ways_make_the_same_calls(monkeypatch):
    gdr.lib()
    assert gdr._quick is not None
    a = calls()
    monkeypatch.setattr(gdr, "_quick", None)
    b = calls()
    for i, (u, v) in enumerate(zip(a, b)):
        assert len(u) == len(v), i
        for s, t in zip(u, v):
            assert (s is None and t is None) or (s.dtype == t.dtype and s.shape == t.shape and torch.equal(s, t)), i


def test_refusals_are_the_same(way):
    e = torch.zeros(2, 1, 6, 4, device="cuda")
    st, i2 = torch.zeros(2, 1, 4, device="cuda"), dev_i32([0, 1])
    cases = [
        (RuntimeError, lambda: gdr.scan_fwd(e.cpu(), e.cpu())),
        (RuntimeError, lambda: gdr.scan_fwd(e, e.cpu())),
        (RuntimeError, lambda: gdr.scan_fwd(e.double(), e.double())),
        (RuntimeError, lambda: gdr.scan_fwd(e.bfloat16(), e.half())),
        (RuntimeError, lambda: gdr.scan_fwd(e.transpose(2, 3), e.transpose(2, 3))),
        (RuntimeError, lambda: gdr.scan_fwd(e, e, st.half())),
        (RuntimeError, lambda: gdr.scan_fwd(e, e, st, i2.long())),
        (ValueError, lambda: gdr.scan_fwd(e[0], e[0])),
        (ValueError, lambda: gdr.scan_fwd(e, e[:, :, :3].contiguous())),
        (ValueError, lambda: gdr.scan_fwd(e, e, st[:1].contiguous())),
        (ValueError, lambda: gdr.scan_fwd(e, e.clone(), out=e)),
        (ValueError, lambda: gdr.scan_fwd(e, e, out=torch.zeros(2, 1, 5, 4, device="cuda"))),
        (RuntimeError, lambda: gdr.scan_fwd(e, None)),
        (ValueError, lambda: gdr.scan_bwd(e, e, torch.zeros(2, 1, 2, 4, device="cuda"), e)),
        (RuntimeError, lambda: gdr.scan_bwd(e, e, None, e)),
        (ValueError, lambda: gdr.scan_step(e, e, st, i2)),
        (ValueError, lambda: gdr.scan_step(e, e, e, torch.zeros(12, dtype=torch.int32, device="cuda"))),
        (ValueError, lambda: gdr.slot_copy([], i2, i2)),
        (ValueError, lambda: gdr.slot_copy([st, st[:1]], i2, i2)),
        (ValueError, lambda: gdr.slot_copy(st, i2, i2[:1])),
        (RuntimeError, lambda: gdr.slot_copy(st.cpu(), i2, i2)),
        (ValueError, lambda: gdr.slot_fork(st, i2, i2.clone(), new_slot_table=i2)),
        (ValueError, lambda: gdr.slot_compact(st, dev_i32([1]))),
        (ValueError, lambda: gdr.slot_free(st, i2.reshape(1, 2))),
        (ValueError, lambda: gdr.conv1d_bwd(torch.zeros(1, 4, 48, device="cuda"), torch.zeros(48, 9, device="cuda"),
                                            *[torch.zeros(1, 1, 4, 16, device="cuda")] * 3)),
        (RuntimeError, lambda: gdr.conv1d_bwd(torch.zeros(1, 4, 48, device="cuda"), torch.zeros(48, 4, device="cuda").half(),
                                              *[torch.zeros(1, 1, 4, 16, device="cuda")] * 3)),
        (RuntimeError, lambda: gdr.scan_fwd(torch.zeros(66, device="cuda")[1:65].reshape(1, 1, 16, 4), e[:1, :, :4].reshape(1, 1, 4, 4)
                                            .repeat(1, 1, 4, 1))),  # not on 16 bytes
    ]
    for k, (err, f) in enumerate(cases):
        with pytest.raises(err):
            f()
    assert gdr.get_error() == 0


def test_marshalling_under_capture_and_on_another_stream(way):
    x, g = torch.randn(1, 2, 50, 16, device="cuda"), -torch.rand(1, 2, 50, 16, device="cuda")
    want = gdr.scan_fwd(x, g)[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gdr.scan_fwd(x, g)[0]
    graph.replay()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        inside = gdr.scan_fwd(x, g)[0]
    other = gdr.scan_fwd(x, g, stream=s)[0]
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(inside, want) and torch.equal(other, want)
