"""The recurrence's kernels in the schedules that large calls take, with strong gates, and with blocks of a cluster that give
up waiting for one another."""
import numpy as np
import pytest
import torch

import gated_deltanet_gdr_b200 as gdr
from oracle import recurrence as R
from tests._bounds import U, check
from tests._helpers import dev, dev_i32, rnd
from tests.test_gpu_scan import draws, lengths_of, run_both, spoil

pytestmark = pytest.mark.gpu


# By the choice of the cut on 148 SMs, for the forward and the backward pass: lanes over the channels, blocks of a cluster
# and tiles.  Every build (vectors of 1, 2 and 4 channels; rows of whole 16 bytes or not; tiles as wide as a warp) takes several
# tiles here, with one block a sequence and with clusters.
SCHEDULES = [
    # rows that are not made of whole 16 bytes: one block a sequence
    (4, 4, 2300, 33, "bf16", "f32", False),   # 4 x 1 x 5, 4 x 1 x 5
    (4, 4, 1100, 33, "f16", "f16", True),     # 4 x 1 x 3, 4 x 1 x 3
    (4, 4, 520, 130, "bf16", "f32", False),   # 8 x 1 x 3, 8 x 1 x 3
    (16, 8, 130, 100, "bf16", "f32", False),  # 16 x 1 x 2, 16 x 1 x 2
    (8, 8, 130, 100, "bf16", "bf16", True),   # 16 x 2 x 1, 16 x 1 x 2
    # and clusters
    (4, 4, 1700, 33, "f32", "f32", True),     # 4 x 2 x 2, 4 x 2 x 2
    (4, 4, 1300, 130, "f16", "f32", True),    # 8 x 2 x 3, 8 x 2 x 3
    (8, 8, 420, 100, "bf16", "f32", True),    # 16 x 2 x 2, 4 x 1 x 1
    (1, 1, 9000, 20, "bf16", "f32", False),   # 4 x 6 x 3, 4 x 6 x 3
    (2, 1, 9000, 34, "f32", "f32", True),     # 4 x 6 x 3, 4 x 6 x 3
    (1, 1, 20001, 7, "f16", "f32", True),     # 4 x 8 x 5, 4 x 8 x 5
    # rows of whole 16 bytes: one block a sequence
    (4, 4, 1100, 132, "f32", "f32", False),   # 4 x 1 x 3, 8 x 1 x 5
    (4, 4, 1100, 260, "f32", "f32", True),    # 8 x 1 x 5, 16 x 1 x 9
    (4, 4, 400, 520, "bf16", "f32", True),    # 16 x 2 x 2, 32 x 1 x 7
    (7, 5, 400, 400, "bf16", "f32", False),   # 32 x 1 x 7, 32 x 1 x 7
    (7, 5, 400, 400, "f16", "f16", True),     # 32 x 1 x 7, 32 x 1 x 7
    (7, 5, 400, 400, "f32", "f32", True),     # 32 x 1 x 7, 32 x 1 x 7
    # and clusters
    (2, 4, 1700, 400, "bf16", "f32", False),  # 32 x 4 x 7, 32 x 4 x 7
    (2, 4, 1700, 400, "f16", "f16", True),    # 32 x 4 x 7, 32 x 4 x 7
    (1, 1, 9000, 16, "bf16", "bf16", True),   # 4 x 6 x 3, 4 x 6 x 3
    (2, 8, 1500, 128, "bf16", "bf16", False),
    (1, 1, 9000, 640, "f16", "f16", True),    # 4 x 6 x 3, 8 x 6 x 6
]


@pytest.mark.parametrize("B,N,S,D,dt,gt,mix", SCHEDULES)
@pytest.mark.parametrize("ragged", [False, True])
def test_several_tiles(B, N, S, D, dt, gt, mix, ragged):
    run_both(B, N, S, D, dt, gt, mix, True, ragged, 800 + S + D)


def strong_bounds(x, g, h0, lengths, mix, dout, dfinal):
    """Bounds before the last rounding, for gates of any strength: (E of every state (B, N, S + 1, D), dx, dg, dinitial).

    Away from 0 a decay is ex2.approx(g log2 e): 2^-22 = 4 u for the function, and its argument carries the constant's and
    the product's rounding, 2 u |g log2 e|, which is 2 u |g| of the result: (4 + 2 |g|) u.  (Near 0 the series loses less.)  A
    result below 2^-126 is 0.  Products, additions and regrouping: 4 u a token, a write of the mixing form 20 u, as in _bounds.
    """
    B, N, S, D = x.shape
    on = (np.arange(S)[None, :] < np.asarray(lengths)[:, None])[:, None, :, None]
    g = np.where(on, g, 0.0)
    a = np.exp(g)
    strong = 8 + 2 * np.where(np.isinf(g), 0.0, np.abs(g))  # e^-inf is 0 exactly
    x, dout = np.where(on, np.abs(x), 0.0), np.where(on, np.abs(dout), 0.0)
    b = (1 - a) * x if mix else x
    lost = 2.0 ** -126
    H, E = [np.abs(h0)], [np.zeros((B, N, D))]
    for t in range(S):
        H.append(a[:, :, t] * H[-1] + b[:, :, t])
        E.append(a[:, :, t] * E[-1] + np.where(on[:, :, t], U * (strong[:, :, t] * H[-1] + 20 * b[:, :, t] * mix) + lost * H[-2], 0.0))
    bx, bg = np.zeros_like(x), np.zeros_like(x)
    mu, e = np.abs(dfinal), np.zeros((B, N, D))
    for t in reversed(range(S)):
        lam, el = dout[:, :, t] + mu, e + U * (dout[:, :, t] + mu)
        w = 1 - a[:, :, t] if mix else np.ones_like(lam)
        bx[:, :, t] = w * el + 20 * U * w * lam * mix
        ok = on[:, :, t]
        mu = np.where(ok, a[:, :, t] * lam, mu)
        e = np.where(ok, a[:, :, t] * el + U * strong[:, :, t] * mu + lost * lam, e)
        diff = H[t] + (x[:, :, t] if mix else 0.0)
        bg[:, :, t] = mu * (E[t] + 3 * U * diff) + diff * e
    return np.stack(E, 2), np.where(on, bx, 0.0), np.where(on, bg, 0.0), e


@pytest.mark.parametrize("mix", [False, True])
@pytest.mark.parametrize("B,N,S,D", [(2, 2, 300, 64), (1, 1, 3000, 33), (7, 5, 150, 400)])
def test_strong_gates(B, N, S, D, mix):
    """Log-decays from -8 to -40 alone, between weak ones, past the smallest fp32 number, and -infinity."""
    x, g, s0, r = draws(B, N, S, D, "f32", "f32", 900 + S)
    s = -r.uniform(8, 40, size=g.shape)
    kind = r.random(size=(1, 1, S, D))
    third = np.arange(D) % 3
    g = np.where((third == 0) | ((third == 1) & (kind < 0.5)), s, g)
    g = np.where((third == 2) & (kind < 0.02), -np.inf, np.where((third == 2) & (kind < 0.05), -100.0, g))
    g = rnd(g, "f32")
    L = lengths_of(B, S, B > 1)
    dout, df = rnd(r.normal(size=x.shape), "f32"), rnd(r.normal(size=(B, N, D)), "f32")
    tx, tg, td = (spoil(dev(v, "f32"), L) for v in (x, g, dout))
    out, fin, ck = gdr.scan_fwd(tx, tg, dev(s0, "f32"), dev_i32(L), mix=mix, output_checkpoints=True)
    dx, dg, di = gdr.scan_bwd(tx, tg, ck, td, dev(df, "f32"), dev_i32(L), mix=mix)
    assert gdr.get_error() == 0
    ro, rf, _ = R.scan_fwd(x, g, s0, L, mix)
    rx, rg, ri = R.scan_bwd(x, g, s0, dout, df, L, mix)
    E, bx, bg, bi = strong_bounds(x, g, s0, L, mix, dout, df)
    check(out, ro, E[:, :, 1:], "f32", "out")
    check(fin, rf, E[:, :, -1], "f32", "final_state")
    check(dx, rx, bx, "f32", "dx")
    check(dg, rg, bg, "f32", "dg")
    check(di, ri, bi, "f32", "dinitial_state")


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
