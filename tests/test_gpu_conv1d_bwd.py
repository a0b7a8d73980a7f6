"""The conv1d's gradient (conv1d_bwd) on the GPU against its fp64 definition.

Bounds, with u = 2^-24: pre is a sum of K + 1 terms, off by d1 = (K + 1) u (|bias| + sum |w x|); s = 1 / (1 + e^{-pre}) is
good to 6 u and silu' = s (1 + pre (1 - s)) to (12 + 8 |pre|) u; its slope is at most 1/2.  So dpre is off by
e = |dy| (d1 / 2 + (12 + 8 |pre|) u).  dx: sum |w| e plus (K + 1) u of the absolute sum.  dweight, dbias: sum |x| e plus one
u of the absolute sum for each addition on the way: at most 128 in a thread, 4 over a block's warps, one for each 32nd of the
blocks' sums and 6 more.
"""
import numpy as np
import pytest
import torch

import gated_deltanet_gdr_b200 as gdr
from oracle import recurrence as R
from tests._bounds import U, check
from tests._helpers import TORCH_DT, dev, dev_i32, host, rnd

pytestmark = pytest.mark.gpu


def split(y, Nk, Nv, Dk, Dv):
    B, S, _ = y.shape
    heads = lambda v, n, d: np.ascontiguousarray(v.reshape(B, S, n, d).transpose(0, 2, 1, 3))
    q = Nk * Dk
    return heads(y[:, :, :q], Nk, Dk), heads(y[:, :, q:2 * q], Nk, Dk), heads(y[:, :, 2 * q:], Nv, Dv)


def draws(B, S, C, K, dt, seed, bias=True, state=True):
    r = np.random.default_rng(seed)
    n = lambda *s, k=1.0: rnd(k * r.normal(size=s), dt)
    return (n(B, S, C), n(C, K, k=0.5), n(C, k=0.2) if bias else None, n(B, C, K) if state else None, n(B, S, C),
            n(B, C, K) if state else None)


def bounds(x, w, bias, state, lengths, dy):
    """bounds of dx, dweight, dbias, dstate before their last rounding"""
    B, S, C = x.shape
    K = w.shape[1]
    bx, bw, bb, bs = np.zeros((B, S, C)), np.zeros((C, K)), np.zeros(C), np.zeros((B, C, K))
    adds = (128 + 4 + 6 + -(-B * -(-max(S, 1) // 64) // 32)) * U  # a block has at least 64 tokens
    for b in range(B):
        L = int(lengths[b])
        hist = np.zeros((K + L, C))
        if state is not None:
            hist[:K] = state[b].T
        hist[K:] = x[b, :L]
        e_hist = np.zeros_like(hist)
        for t in range(L):
            win = hist[t + 1:t + 1 + K]
            wx, bi = (np.abs(w.T) * np.abs(win)).sum(0), 0.0 if bias is None else bias
            pre = (w.T * win).sum(0) + bi
            s = 1 / (1 + np.exp(-pre))
            d = np.abs(dy[b, t] * (s + pre * s * (1 - s)))
            e = np.abs(dy[b, t]) * ((K + 1) * U * (wx + np.abs(bi)) / 2 + (12 + 8 * np.abs(pre)) * U)
            e_hist[t + 1:t + 1 + K] += np.abs(w.T) * (e + (K + 1) * U * d)
            bw += (np.abs(win) * (e + (adds + U) * d)).T
            bb += e + adds * d
        bx[b, :L] = e_hist[K:]
        bs[b] = e_hist[:K].T
    # the new state's gradient is one more addition
    return bx, bw, bb, bs


def one(B, S, Nk, Nv, Dk, Dv, K, dt, lengths=None, seed=0, bias=True, state=True):
    C = 2 * Nk * Dk + Nv * Dv
    x, w, bi, st, dy, ds = draws(B, S, C, K, dt, seed, bias, state)
    L = np.full(B, S) if lengths is None else np.asarray(lengths)
    tx = dev(x, dt)
    tq, tk, tv = (dev(v, dt) for v in split(dy, Nk, Nv, Dk, Dv))
    for b in range(B):  # padding holds anything
        tx[b, int(L[b]):] = float("nan")
        for t in (tq, tk, tv):
            t[b, :, int(L[b]):] = float("inf")
    got = gdr.conv1d_bwd(tx, dev(w, dt), tq, tk, tv, dev(bi, dt), dev(st, dt), dev_i32(lengths), dev(ds, dt))
    assert gdr.get_error() == 0
    want = R.conv1d_bwd(x, w, bi, st, L, dy, ds)
    bx, bw, bb, bs = bounds(x, w, bi, st, L, dy)
    last = U * (np.abs(want[0]) + bx), U * (np.abs(want[3]) + bs)
    check(got[0], want[0], bx + last[0], dt, "dx")
    check(got[1], want[1], bw, "f32", "dweight")
    check(got[2], want[2], bb, "f32", "dbias")
    check(got[3], want[3], bs + last[1], dt, "dconv_state")
    return got


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("K", [1, 2, 3, 4, 5, 6, 7, 8])
def test_taps_and_types(dt, K):
    one(2, 70, 1, 2, 32, 16, K, dt, [70, 33], 10 + K)


@pytest.mark.parametrize("S", [1, 2, 3, 63, 64, 65, 67, 255, 256, 257, 259, 600])
def test_lengths_at_the_tiles_ends(S):
    one(4, S, 1, 1, 16, 32, 4, "f32", [S, max(0, S - 1), min(S, 2), 0], 40 + S)
    one(1, S, 1, 1, 16, 32, 8, "bf16", None, 60 + S, bias=False, state=False)


@pytest.mark.parametrize("Nk,Nv,Dk,Dv", [(1, 1, 16, 16), (2, 6, 64, 32), (1, 2, 128, 128), (3, 3, 16, 128)])
def test_heads(Nk, Nv, Dk, Dv):
    one(2, 130, Nk, Nv, Dk, Dv, 4, "f32", None, 80 + Dk)


def test_many_sequences_and_equal_bits():
    a = one(70, 20, 1, 1, 16, 16, 3, "bf16", [20 * b // 69 for b in range(70)], 90)
    b = one(70, 20, 1, 1, 16, 16, 3, "bf16", [20 * b // 69 for b in range(70)], 90)
    for u, v in zip(a, b):
        assert torch.equal(u, v)


def test_large_preactivations():
    """silu' far out: 1 on the right, 0 on the left, without NaN."""
    x = torch.tensor([300.0, -300.0, 88.0, -88.0, -104.0, 0.0], device="cuda").repeat(8).reshape(1, 48, 1).expand(1, 48, 48)
    x = x.contiguous()
    w = torch.ones(48, 1, device="cuda")
    one_ = torch.ones(1, 1, 48, 16, device="cuda")
    dx, dw, db, _ = gdr.conv1d_bwd(x, w, one_, one_, one_)
    p = host(x)
    s = 1 / (1 + np.exp(-p))
    want = s + p * s * (1 - s)
    assert np.abs(host(dx) - want).max() <= 200 * U  # |silu'| <= 1.1, off by (12 + 8 |p|) u where s is neither 0 nor 1
    assert torch.isfinite(dw).all() and torch.isfinite(db).all()


def test_no_tokens_and_no_sequences():
    w = torch.ones(48, 4, device="cuda")
    z = torch.empty(2, 1, 0, 16, device="cuda")
    ds = torch.randn(2, 48, 4, device="cuda")
    dx, dw, db, d = gdr.conv1d_bwd(torch.empty(2, 0, 48, device="cuda"), w, z, z, z, None, ds.clone(), None, ds)
    assert dx.numel() == 0 and not torch.any(dw) and not torch.any(db) and torch.equal(d, ds)
    z = torch.empty(0, 1, 5, 16, device="cuda")
    dx, dw, db, d = gdr.conv1d_bwd(torch.empty(0, 5, 48, device="cuda"), w, z, z, z)
    assert not torch.any(dw) and not torch.any(db)


def test_bad_length_contributes_nothing():
    x, w, bi, st, dy, ds = draws(3, 40, 48, 4, "f32", 5)
    t = [dev(v, "f32") for v in split(dy, 1, 1, 16, 16)]
    got = gdr.conv1d_bwd(dev(x, "f32"), dev(w, "f32"), *t, dev(bi, "f32"), dev(st, "f32"), dev_i32([40, 41, 7]),
                         dev(ds, "f32"))
    assert gdr.get_error() == gdr.DEVERR_LENGTH
    assert not torch.any(got[0][1]) and not torch.any(got[3][1])
    k = [0, 2]
    want = R.conv1d_bwd(x[k], w, bi, st[k], np.array([40, 7]), dy[k], ds[k])
    _, bw, bb, _ = bounds(x[k], w, bi, st[k], [40, 7], dy[k])
    check(got[1], want[1], bw, "f32", "dweight")
    check(got[2], want[2], bb, "f32", "dbias")


def test_graph_and_side_stream_with_a_workspace():
    x, w, bi, st, dy, ds = draws(2, 300, 96, 4, "bf16", 6)
    t = [dev(v, "bf16") for v in split(dy, 1, 2, 16, 32)]
    args = [dev(x, "bf16"), dev(w, "bf16"), *t, dev(bi, "bf16"), dev(st, "bf16"), None, dev(ds, "bf16")]
    want = gdr.conv1d_bwd(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gdr.conv1d_bwd(*args, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    ws = torch.empty(gdr.conv1d_bwd_workspace_bytes(2, 300, 1, 2, 16, 32, 4), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = gdr.conv1d_bwd(*args, workspace=ws)
    graph.replay()
    for u, v, z in zip(got, want, g):
        assert torch.equal(u, v) and torch.equal(z, v)


def test_refusals():
    x, w = torch.zeros(1, 4, 48, device="cuda"), torch.zeros(48, 4, device="cuda")
    d = torch.zeros(1, 1, 4, 16, device="cuda")
    with pytest.raises(ValueError):
        gdr.conv1d_bwd(x, w, d, d, torch.zeros(1, 1, 4, 32, device="cuda"))
    with pytest.raises(ValueError):
        gdr.conv1d_bwd(x, w, d, torch.zeros(1, 1, 3, 16, device="cuda"), d)
    with pytest.raises(RuntimeError):
        gdr.conv1d_bwd(x, w.half(), d, d, d)
    with pytest.raises(ValueError):
        gdr.conv1d_bwd(x, torch.zeros(48, 9, device="cuda"), d, d, d)
    with pytest.raises(ValueError):
        gdr.conv1d_bwd(x, w, d, d, d, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        gdr.conv1d_bwd(x, w, d, d, d, dx=x)
    with pytest.raises(RuntimeError):
        gdr.conv1d_bwd(torch.zeros(1, 4, 36, device="cuda"), torch.zeros(36, 4, device="cuda"),
                       *[torch.zeros(1, 1, 4, 12, device="cuda")] * 3)
