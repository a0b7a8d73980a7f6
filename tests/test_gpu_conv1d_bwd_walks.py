"""The conv1d's gradient behind the end of a sequence, and in the walks that large calls take.

Bounds as in test_gpu_conv1d_bwd: the sums of dweight and dbias take at most 128 additions in a thread."""
import numpy as np
import pytest
import torch

import gated_deltanet_gdr_b200 as gdr
from oracle import recurrence as R
from tests._bounds import U, check
from tests._helpers import dev, dev_i32, host
from tests.test_gpu_conv1d_bwd import bounds, draws, split

pytestmark = pytest.mark.gpu

ENDS = [0, 1, 2, 3, 7, 8, 9, 15, 16, 17, 31, 33, 64, 70]


def call(x, w, bi, st, dy, ds, L, dt, heads, spoil=float("nan")):
    tx, t = dev(x, dt), [dev(v, dt) for v in split(dy, *heads)]
    for b in range(x.shape[0]):
        tx[b, int(L[b]):] = spoil
        for v in t:
            v[b, :, int(L[b]):] = spoil
    got = gdr.conv1d_bwd(tx, dev(w, dt), *t, dev(bi, dt), dev(st, dt), dev_i32(L), dev(ds, dt))
    assert gdr.get_error() == 0
    return got


@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("K", [2, 4, 8])
def test_products_that_overflow_behind_the_end_only(K, state):
    """The last input times the first tap overflows, which only the padding's windows would hold: every gradient is finite."""
    heads, S, B = (1, 1, 16, 16), 70, len(ENDS)
    x, w, bi, st, dy, ds = draws(B, S, 48, K, "f32", 20 + K, state=state)
    w[5] = 0.0
    w[5, 0] = 2.0 ** 66
    w[21, 0], w[21, 1:] = -(2.0 ** 66), 0.0
    for b, L in enumerate(ENDS):
        if L:
            x[b, L - 1, [5, 21]] = 2.0 ** 100
    # the valid windows of those channels hold the large tap against ordinary inputs: pre is 0 or far out, where silu' is 0 or 1
    got = call(x, w, bi, st, dy, ds, ENDS, "f32", heads)
    want = R.conv1d_bwd(x, w, bi, st, np.array(ENDS), dy, ds)
    for u, v in zip(got, want):
        assert bool(torch.isfinite(u).all()) and np.isfinite(v).all()
    for b, L in enumerate(ENDS):
        assert not torch.any(got[0][b, L:])
    keep = [c for c in range(48) if c not in (5, 21)]
    bx, bw, bb, bs = bounds(x[..., keep], w[keep], bi[keep], st[:, keep] if state else None, ENDS, dy[..., keep])
    last = U * (np.abs(want[0][..., keep]) + bx), U * (np.abs(want[3][:, keep]) + bs)
    check(got[0][..., keep], want[0][..., keep], bx + last[0], "f32", "dx")
    check(got[1][keep], want[1][keep], bw, "f32", "dweight")
    check(got[2][keep], want[2][keep], bb, "f32", "dbias")
    check(got[3][:, keep], want[3][:, keep], bs + last[1], "f32", "dconv_state")


@pytest.mark.parametrize("dt,value", [("f32", np.inf), ("f32", np.nan), ("bf16", -np.inf), ("f16", np.inf)])
@pytest.mark.parametrize("K", [1, 4, 8])
def test_values_that_are_not_finite_before_the_end(K, dt, value):
    """An infinity in the last valid inputs stays in its channel and in its sequence's valid tokens: padding is zero."""
    heads, S, B = (1, 1, 16, 16), 70, len(ENDS)
    x, w, bi, st, dy, ds = draws(B, S, 48, K, dt, 30 + K)
    clean = call(x, w, bi, st, dy, ds, ENDS, dt, heads)
    y = x.copy()
    for b, L in enumerate(ENDS):
        y[b, max(0, L - 2):L, 11] = value
    got = call(y, w, bi, st, dy, ds, ENDS, dt, heads, spoil=float("inf"))
    keep = [c for c in range(48) if c != 11]
    for b, L in enumerate(ENDS):
        assert not torch.any(got[0][b, L:])  # (a NaN is not zero)
    assert torch.equal(got[0][..., keep], clean[0][..., keep]) and torch.equal(got[1][keep], clean[1][keep])
    assert torch.equal(got[2][keep], clean[2][keep]) and torch.equal(got[3][:, keep], clean[3][:, keep])
    # an empty sequence passes its state's gradient on, whatever its taps are
    w[11] = np.inf
    got = call(x, w, bi, st, dy, ds, ENDS, dt, heads)
    assert np.array_equal(host(got[3][0]), ds[0]) and not torch.any(got[0][0])
    for b, L in enumerate(ENDS):
        assert not torch.any(got[0][b, L:])


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("K,S,ends", [(4, 1500, [1500, 1027, 511, 130]), (4, 1536, [1536, 1408, 385, 129]),
                                      (8, 1500, [1499, 1025, 512, 64]), (3, 1500, None), (1, 1500, [1500, 1024, 513, 7])])
def test_long_walks(dt, K, S, ends):
    """Walks of 128 tokens a warp (16-bit types) and of 64 (fp32), with ends around theirs: 4 sequences of 4096 channels,
    of which every 61st is compared."""
    heads = (8, 16, 128, 128)
    B, C = 4, 4096
    x, w, bi, st, dy, ds = draws(B, S, C, K, dt, 50 + K + S)
    L = [S] * B if ends is None else ends
    got = call(x, w, bi, st, dy, ds, L, dt, heads)
    c = np.arange(7, C, 61)
    args = x[..., c], w[c], bi[c], st[:, c]
    want = R.conv1d_bwd(*args, np.array(L), dy[..., c], ds[:, c])
    bx, bw, bb, bs = bounds(*args, L, dy[..., c])
    last = U * (np.abs(want[0]) + bx), U * (np.abs(want[3]) + bs)
    check(got[0][..., c], want[0], bx + last[0], dt, "dx")
    check(got[1][c], want[1], bw, "f32", "dweight")
    check(got[2][c], want[2], bb, "f32", "dbias")
    check(got[3][:, c], want[3], bs + last[1], dt, "dconv_state")
    for b in range(B):
        assert not torch.any(got[0][b, L[b]:])
