"""Pins of the fp64 definitions in oracle/recurrence.py: closed forms, a scan by doubling, differences, invariants."""
import numpy as np
import pytest

import oracle
from oracle import recurrence as R


def case(B=2, N=2, S=9, D=3, seed=0):
    r = np.random.default_rng(seed)
    return r.normal(size=(B, N, S, D)), -np.exp(r.normal(size=(B, N, S, D)) - 1), r.normal(size=(B, N, D)), r


@pytest.mark.parametrize("mix", [False, True])
def test_constant_decay_is_geometric(mix):
    a, x0, h0 = 0.75, 1.5, -2.0
    S = 12
    x, g = np.full((1, 1, S, 1), x0), np.full((1, 1, S, 1), np.log(a))
    out, fin, _ = R.scan_fwd(x, g, np.full((1, 1, 1), h0), None, mix)
    for t in range(S):
        b = (1 - a) * x0 if mix else x0
        want = a ** (t + 1) * h0 + b * (1 - a ** (t + 1)) / (1 - a)
        assert abs(out[0, 0, t, 0] - want) < 1e-13
    assert fin[0, 0, 0] == out[0, 0, -1, 0]


def test_scan_equals_the_scan_by_doubling():
    """The recurrence's composition (a2 a1, a2 b1 + b2) is associative: the inclusive scan by doubled spans."""
    x, g, h0, _ = case(S=37)
    out, _, _ = R.scan_fwd(x, g, h0)
    a, b = np.exp(g), x.copy()
    b[:, :, 0] += a[:, :, 0] * h0
    d = 1
    while d < 37:
        b[:, :, d:] = b[:, :, d:] + a[:, :, d:] * b[:, :, :-d]
        a[:, :, d:] = a[:, :, d:] * a[:, :, :-d]
        d *= 2
    assert np.abs(out - b).max() < 1e-12


def test_split_lengths_checkpoints_and_forgetting():
    x, g, h0, r = case(B=3, S=150)
    lengths = np.array([150, 70, 0])
    out, fin, ck = R.scan_fwd(x, g, h0, lengths)
    o1, f1, _ = R.scan_fwd(x[:, :, :64], g[:, :, :64], h0, np.minimum(lengths, 64))
    o2, f2, _ = R.scan_fwd(x[:, :, 64:], g[:, :, 64:], f1, np.maximum(lengths - 64, 0))
    assert np.array_equal(np.concatenate([o1, o2], 2), out) and np.array_equal(f2, fin)
    assert np.array_equal(ck[:, :, 0], h0) and np.array_equal(ck[:2, :, 1], f1[:2])
    assert np.all(out[1, :, 70:] == 0) and np.array_equal(fin[2], h0[2])
    g[:, :, 40] = -np.inf  # a boundary: nothing before it counts
    a, _, _ = R.scan_fwd(x, g, h0, lengths)
    b, _, _ = R.scan_fwd(x[:, :, 40:], g[:, :, 40:], None, np.maximum(lengths - 40, 0))
    assert np.array_equal(a[:, :, 40:], b)


def test_mix_of_a_constant_keeps_it():
    _, g, _, _ = case(S=20)
    x = np.full(g.shape, 3.25)
    out, _, _ = R.scan_fwd(x, g, np.full((2, 2, 3), 3.25), None, True)
    assert np.abs(out - 3.25).max() < 1e-14


@pytest.mark.parametrize("mix", [False, True])
def test_scan_gradient_against_differences(mix):
    x, g, h0, r = case(S=7)
    lengths = np.array([7, 4])
    dout, dfin = r.normal(size=x.shape), r.normal(size=h0.shape)
    loss = lambda x, g, h0: sum((u * v).sum() for u, v in zip(R.scan_fwd(x, g, h0, lengths, mix)[:2], (dout, dfin)))
    grads = R.scan_bwd(x, g, h0, dout, dfin, lengths, mix)
    e = 1e-6
    for k, got in enumerate(grads):
        args = [x, g, h0]
        for at in list(np.ndindex(args[k].shape))[::5]:
            hi, lo = [a.copy() for a in args], [a.copy() for a in args]
            hi[k][at] += e
            lo[k][at] -= e
            num = (loss(*hi) - loss(*lo)) / (2 * e)
            assert abs(num - got[at]) < 1e-6 * max(1.0, abs(num)), (k, at)  # e^2 f''' / 6 and 2^-53 |loss| / e


def test_step_equals_the_scan():
    x, g, h0, r = case(B=2, S=5)
    pool = r.normal(size=(6, 2, 3))
    out, fin, _ = R.scan_fwd(x, g, pool[[4, 1]])
    o, p = R.scan_step(x, g, pool, [4] * 5 + [1] * 5)
    assert np.array_equal(o, out) and np.array_equal(p[[4, 1]], fin)
    assert np.array_equal(p[[0, 2, 3, 5]], pool[[0, 2, 3, 5]])
    # accepted counts: outputs of all tokens, state after the accepted ones
    o, p = R.scan_step(x, g, pool, [4] * 5 + [1] * 5, None, [2, 0])
    assert np.array_equal(o, out) and np.array_equal(p[4], out[0, :, 1]) and np.array_equal(p[1], pool[1])
    # a slot per token: the next step goes on from the accepted token's slot
    pool = r.normal(size=(11, 2, 3))
    idx = np.arange(10)
    o1, p1 = R.scan_step(x, g, pool, idx, None, None, False, True)
    o2, _ = R.scan_step(x[:, :, :1], g[:, :, :1], p1, [2, 8], None, None)
    w, _, _ = R.scan_fwd(np.concatenate([x[:, :, :3], x[:, :, :1]], 2), np.concatenate([g[:, :, :3], g[:, :, :1]], 2),
                         pool[[0, 5]])
    w1, _, _ = R.scan_fwd(np.concatenate([x[:, :, :4], x[:, :, :1]], 2), np.concatenate([g[:, :, :4], g[:, :, :1]], 2),
                          pool[[0, 5]])
    assert np.array_equal(o2[0], w[0, :, 3:]) and np.array_equal(o2[1], w1[1, :, 4:])


@pytest.mark.parametrize("K", [1, 3, 4])
def test_conv_gradient_against_differences_of_the_conv(K):
    r = np.random.default_rng(K)
    B, S, C = 3, 6, 4
    x, w, bias, st = r.normal(size=(B, S, C)), r.normal(size=(C, K)), r.normal(size=C), r.normal(size=(B, C, K))
    lengths = np.array([6, 2, 0], np.int32)
    dy, ds = r.normal(size=(B, S, C)), r.normal(size=(B, C, K))
    loss = lambda x, w, bias, st: sum((u * v).sum() for u, v in zip(oracle.causal_conv1d(x, w, bias, st, lengths), (dy, ds)))
    grads = R.conv1d_bwd(x, w, bias, st, lengths, dy, ds)
    e = 1e-6
    for k, got in enumerate(grads):
        args = [x, w, bias, st]
        for at in list(np.ndindex(args[k].shape))[::3]:
            hi, lo = [a.copy() for a in args], [a.copy() for a in args]
            hi[k][at] += e
            lo[k][at] -= e
            num = (loss(*hi) - loss(*lo)) / (2 * e)
            assert abs(num - got[at]) < 1e-6 * max(1.0, abs(num)), (k, at)


def test_fork_keeps_every_row_its_parents_state_with_the_fewest_copies():
    r = np.random.default_rng(3)
    for n in (1, 2, 7, 40):
        pools = [r.normal(size=(n + 3, 2)), r.integers(0, 9, size=(n + 3, 5))]
        table = r.permutation(n + 3)[:n].astype(np.int32)
        parents = r.integers(0, n, size=n)
        res, new, bad = R.slot_fork(pools, table, parents)
        assert not bad and sorted(new) == sorted(table)
        for p, q in zip(pools, res):
            assert np.array_equal(q[new], p[table[parents]])
            changed = {i for i in range(n + 3) if not np.array_equal(p[i], q[i])}
            assert len(changed) <= n - len(set(parents)) and changed <= set(table)


def test_compact_and_copy_and_free():
    r = np.random.default_rng(4)
    pools = [r.normal(size=(9, 4))]
    live = np.array([0, 1, 0, 0, 1, 1, 0, 1, 1], np.int32)
    res, new, n = R.slot_compact(pools, live)
    assert n == 5 and list(new) == [-1, 1, -1, -1, 4, 0, -1, 2, 3]
    for s in range(9):
        if live[s]:
            assert np.array_equal(res[0][new[s]], pools[0][s])
    assert np.array_equal(res[0][5:], pools[0][5:])
    res, bad = R.slot_copy(pools, [1, 1, -1, 4, 4], [2, 3, 0, -1, 4])
    assert not bad and np.array_equal(res[0][[2, 3]], pools[0][[1, 1]]) and np.array_equal(res[0][0], pools[0][0])
    res, bad = R.slot_copy(pools, [1, 2, 5, 6, 9], [2, 3, 7, 7, 8])  # 2 is a source, 7 is named twice, 9 is no slot
    assert bad and np.array_equal(res[0][2], pools[0][2]) and np.array_equal(res[0][3], pools[0][2])
    assert np.array_equal(res[0][7], pools[0][5]) and np.array_equal(res[0][8], pools[0][8])
    res, lv, bad = R.slot_free(pools, [3, -1, 3, 9], np.ones(9, np.int32))
    assert bad and np.all(res[0][3] == 0) and lv.sum() == 8
