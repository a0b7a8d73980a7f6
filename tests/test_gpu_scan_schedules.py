"""The recurrence's kernels in the schedules that large calls take: blocks of a cluster that give up waiting for one another."""
import pytest
import torch

import gated_deltanet_gdr_b200 as gdr
from tests._helpers import dev, dev_i32
from tests.test_gpu_scan import draws

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,N,S,D,dt,mix", [(1, 1, 6000, 64, "f32", False), (1, 1, 9000, 640, "f16", True),
                                            (7, 5, 777, 100, "f32", True), (1, 1, 20001, 7, "bf16", False),
                                            (3, 1, 5000, 130, "bf16", True), (2, 8, 3000, 128, "bf16", False)])
def test_waits_that_run_out_leave_nothing_behind(B, N, S, D, dt, mix):
    """Limits from one that the first test of a wait is over at to one that some waits keep: every call ends with the flag or
    with the right outputs, whatever tile its blocks give up at, and so does the next one at once."""
    x, g, s0, _ = draws(B, N, S, D, dt, "f32", 700 + D)
    tx, tg, st = dev(x, dt), dev(g, "f32"), dev(s0, "f32")
    lens = dev_i32([S, 0, max(1, S // 2), S, S, 1, S][:B])
    want = gdr.scan_fwd(tx, tg, st, lens, mix=mix, output_checkpoints=True)
    wg = gdr.scan_bwd(tx, tg, want[2], tx, st, lens, mix=mix)
    assert gdr.get_error() == 0
    flagged = 0
    try:
        for ns in [1] * 8 + [1100, 1500, 2000, 3000, 5000, 8000] * 3:
            gdr.set_wait_limit_ns(ns)
            o = gdr.scan_fwd(tx, tg, st, lens, mix=mix)
            e = gdr.get_error()
            assert e in (0, gdr.DEVERR_TIMEOUT)
            assert e or (torch.equal(o[0], want[0]) and torch.equal(o[1], want[1]))
            b = gdr.scan_bwd(tx, tg, want[2], tx, st, lens, mix=mix)
            f = gdr.get_error()
            assert f in (0, gdr.DEVERR_TIMEOUT)
            assert f or all(torch.equal(u, v) for u, v in zip(b, wg))
            flagged += bool(e) + bool(f)
    finally:
        gdr.set_wait_limit_ns(0)
    assert flagged > 0
    for _ in range(3):
        o = gdr.scan_fwd(tx, tg, st, lens, mix=mix)
        b = gdr.scan_bwd(tx, tg, want[2], tx, st, lens, mix=mix)
        assert all(torch.equal(u, v) for u, v in zip(o[:2] + b, want[:2] + wg))
    assert gdr.get_error() == 0
