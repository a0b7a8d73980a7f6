"""The gated linear recurrence (scan_fwd, scan_bwd, scan_step) on the GPU against its fp64 definition."""
import numpy as np
import pytest
import torch

import gated_deltanet_gdr_b200 as gdr
from oracle import recurrence as R
from tests._bounds import bwd_bounds, check, scan_bounds
from tests._helpers import TORCH_DT, dev, dev_i32, host, rnd

pytestmark = pytest.mark.gpu

TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")]


def draws(B, N, S, D, dt, gt, seed, h0=True):
    """inputs as the call sees them (rounded), in fp64; rates from memories of a token to a few hundred"""
    r = np.random.default_rng(seed)
    x = rnd(r.normal(size=(B, N, S, D)), dt)
    rate = np.exp(r.uniform(np.log(5e-3), np.log(2.0), size=D))
    g = rnd(-rate * np.log1p(np.exp(r.normal(size=(B, N, S, D)))), gt)
    return x, g, (rnd(r.normal(size=(B, N, D)), "f32") if h0 else None), r


def lengths_of(B, S, ragged):
    return np.array([S * b // max(B - 1, 1) for b in range(B)] if ragged else [S] * B, np.int32)


def spoil(t, lengths, value=float("nan")):
    """padding of a device tensor (B, N, S, D) set to NaN"""
    for b, L in enumerate(lengths):
        t[b, :, int(L):] = value
    return t


def run_both(B, N, S, D, dt, gt, mix, h0, ragged, seed, dfinal=True):
    x, g, s0, r = draws(B, N, S, D, dt, gt, seed, h0)
    L = lengths_of(B, S, ragged)
    dout, df = rnd(r.normal(size=x.shape), dt), rnd(r.normal(size=(B, N, D)), "f32") if dfinal else None
    tx, tg, td = (spoil(dev(v, t), L) for v, t in ((x, dt), (g, gt), (dout, dt)))
    lens = dev_i32(L) if ragged else None
    out, fin, ck = gdr.scan_fwd(tx, tg, dev(s0, "f32"), lens, mix=mix, output_checkpoints=True)
    grads = gdr.scan_bwd(tx, tg, ck, td, dev(df, "f32"), lens, mix=mix)
    assert gdr.get_error() == 0
    ro, rf, rc = R.scan_fwd(x, g, s0, L, mix)
    E, H = scan_bounds(x, g, s0, L, mix)
    check(out, ro, E[:, :, 1:], dt, "out")
    check(fin, rf, E[:, :, -1], "f32", "final_state")
    for b in range(B):
        n = max(1, -(-int(L[b]) // 64))
        check(ck[b, :, :n], rc[b, :, :n], E[b, :, :64 * n:64][:, :n], "f32", "checkpoints")
        assert not torch.any(out[b, :, int(L[b]):]) and not torch.any(grads[0][b, :, int(L[b]):])
        assert not torch.any(grads[1][b, :, int(L[b]):])
        if L[b] == 0:
            assert np.array_equal(host(fin[b]), np.zeros((N, D)) if s0 is None else s0[b])
            assert np.array_equal(host(grads[2][b]), np.zeros((N, D)) if df is None else df[b])
    first = np.zeros((B, N, D)) if s0 is None else s0
    h = np.concatenate([first[:, :, None], ro], 2)
    bx, bg, bi = bwd_bounds(x, g, s0, L, mix, dout, df, E, H, h)
    rx, rg, ri = R.scan_bwd(x, g, s0, dout, df, L, mix)
    check(grads[0], rx, bx, dt, "dx")
    check(grads[1], rg, bg, gt, "dg")
    check(grads[2], ri, bi, "f32", "dinitial_state")
    return (out, fin, ck) + grads


@pytest.mark.parametrize("dt,gt", TYPES)
@pytest.mark.parametrize("mix", [False, True])
@pytest.mark.parametrize("S", [1, 2, 63, 64, 65, 130, 600])
def test_scan_and_gradient(dt, gt, mix, S):
    run_both(3, 2, S, 40, dt, gt, mix, True, True, 10 + S)


@pytest.mark.parametrize("D", [1, 3, 4, 7, 31, 64, 100, 128, 130, 132, 260, 1000, 1028])
def test_channel_counts(D):
    """Rows whose length is no multiple of a vector, of a warp or of a block's channels."""
    run_both(2, 1 if D > 300 else 3, 150, D, "bf16", "f32", False, True, True, 100 + D)
    run_both(2, 1, 70, D, "f32", "f32", True, False, False, 200 + D, dfinal=False)
    run_both(1, 2, 70, D, "f16", "f16", True, True, False, 300 + D)


@pytest.mark.parametrize("B,N,S,D", [(1, 1, 5000, 16), (1, 1, 2049, 256), (2, 1, 1023, 512), (40, 9, 33, 128),
                                     (1, 40, 513, 128), (300, 1, 3, 64), (5, 1, 700, 2048)])
def test_few_chains_and_many(B, N, S, D):
    """One long sequence (split over time), and more chains than the GPU holds at once."""
    run_both(B, N, S, D, "bf16", "bf16", True, True, B > 1, 400 + S)


def test_equal_calls_give_equal_bits():
    a = run_both(2, 2, 1500, 96, "bf16", "f32", False, True, False, 500)
    b = run_both(2, 2, 1500, 96, "bf16", "f32", False, True, False, 500)
    for u, v in zip(a, b):
        assert torch.equal(u, v)


def test_forgetting_gate_and_values_that_are_not_finite():
    """g = -inf forgets what was there; an infinity or NaN stays in its own channel and after its own token."""
    x, g, s0, _ = draws(1, 2, 300, 128, "f32", "f32", 520)
    g[:, :, 100] = -np.inf
    x2 = x.copy()
    x2[0, 0, 200, 5], x2[0, 1, 250, 127] = np.inf, np.nan
    out, fin, _ = gdr.scan_fwd(dev(x2, "f32"), dev(g, "f32"), dev(s0, "f32"))
    ro, rf, _ = R.scan_fwd(x, g, s0)
    E, _ = scan_bounds(x, g, s0, [300], False)
    o = host(out)
    assert np.isposinf(o[0, 0, 200, 5]) and not np.any(np.isfinite(o[0, 0, 200:, 5]))
    assert np.all(np.isnan(o[0, 1, 250:, 127]))
    o[0, 0, 200:, 5], o[0, 1, 250:, 127] = ro[0, 0, 200:, 5], ro[0, 1, 250:, 127]
    check(o, ro, E[:, :, 1:], "f32", "out")
    assert np.array_equal(o[:, :, 100], rnd(x, "f32")[:, :, 100])


def test_nothing_decays_and_everything_does():
    """g = 0 sums the inputs (exact for small whole numbers); g = -200 leaves the input alone."""
    r = np.random.default_rng(7)
    x = r.integers(-8, 9, size=(1, 1, 4097, 12)).astype(np.float64)
    out, fin, _ = gdr.scan_fwd(dev(x, "f32"), torch.zeros(1, 1, 4097, 12, device="cuda"))
    assert np.array_equal(host(out), np.cumsum(x, 2)) and np.array_equal(host(fin), x.sum(2))
    out, _, _ = gdr.scan_fwd(dev(x, "f32"), torch.full((1, 1, 4097, 12), -200.0, device="cuda"))
    assert np.array_equal(host(out), x)


def test_in_place_state_split_calls_and_no_state():
    """Two calls that hand the state on in place equal one; a call may leave out the final state."""
    x, g, s0, _ = draws(2, 3, 200, 36, "bf16", "f32", 530)
    tx, tg, st = dev(x, "bf16"), dev(g, "f32"), dev(s0, "f32")
    whole, fin, _ = gdr.scan_fwd(tx, tg, st.clone())
    cut = 77
    o1, s1, none = gdr.scan_fwd(tx[:, :, :cut].contiguous(), tg[:, :, :cut].contiguous(), st, final_state=st)
    assert s1 is st and none is None
    o2, s2, _ = gdr.scan_fwd(tx[:, :, cut:].contiguous(), tg[:, :, cut:].contiguous(), st, final_state=st)
    ro, rf, _ = R.scan_fwd(x, g, s0)
    E, _ = scan_bounds(x, g, s0, [200, 200], False)
    check(torch.cat([o1, o2], 2), ro, E[:, :, 1:], "bf16", "out")
    check(st, rf, E[:, :, -1], "f32", "state")
    check(whole, ro, E[:, :, 1:], "bf16", "whole")
    o, f, _ = gdr.scan_fwd(tx, tg, None, output_final_state=False)
    assert f is None and gdr.get_error() == 0


def test_no_tokens():
    st = torch.randn(2, 3, 8, device="cuda")
    e = torch.empty(2, 3, 0, 8, device="cuda")
    out, fin, _ = gdr.scan_fwd(e, e, st)
    assert out.shape == e.shape and torch.equal(fin, st)
    _, fin, _ = gdr.scan_fwd(e, e)
    assert not torch.any(fin)
    dx, dg, di = gdr.scan_bwd(e, e, torch.empty(2, 3, 0, 8, device="cuda"), e, st)
    assert torch.equal(di, st)


def test_bad_length_is_skipped_and_flagged():
    x, g, s0, _ = draws(3, 2, 90, 20, "f32", "f32", 540)
    tx, tg, st = dev(x, "f32"), dev(g, "f32"), dev(s0, "f32")
    for bad in (-1, 91):
        lens = dev_i32([90, bad, 17])
        fin = torch.full_like(st, 7.0)
        ck = torch.full(gdr.scan_checkpoint_shape(3, 2, 90, 20), 9.0, device="cuda")
        out, _, _ = gdr.scan_fwd(tx, tg, st, lens, final_state=fin, checkpoints=ck)
        assert gdr.get_error() == gdr.DEVERR_LENGTH
        assert not torch.any(out[1]) and bool((fin[1] == 7).all()) and bool((ck[1] == 9).all())
        assert bool((ck[2, :, 1:] == 9).all())  # chunks behind the last token are left as they were
        ro, rf, _ = R.scan_fwd(x, g, s0, [90, 0, 17])
        E, _ = scan_bounds(x, g, s0, [90, 0, 17], False)
        check(out, ro, E[:, :, 1:], "f32", "out")
        dx, dg, di = gdr.scan_bwd(tx, tg, ck, tx, st, lens)
        assert gdr.get_error() == gdr.DEVERR_LENGTH
        assert not torch.any(dx[1]) and not torch.any(dg[1]) and not torch.any(di[1])


def test_side_stream_and_graph():
    """A call on a stream of its own, and forward and backward captured together and replayed on new inputs."""
    x, g, s0, r = draws(2, 2, 700, 128, "bf16", "f32", 550)
    tx, tg, st = dev(x, "bf16"), dev(g, "f32"), dev(s0, "f32")
    want = gdr.scan_fwd(tx, tg, st, output_checkpoints=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gdr.scan_fwd(tx, tg, st, output_checkpoints=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for u, v in zip(got, want):
        assert torch.equal(u, v)
    dout = torch.randn_like(tx)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, f, c = gdr.scan_fwd(tx, tg, st, output_checkpoints=True)
        grads = gdr.scan_bwd(tx, tg, c, dout, f)
    for seed in (1, 2):
        torch.manual_seed(seed)
        tx.normal_()
        dout.normal_()
        graph.replay()
        w = gdr.scan_fwd(tx, tg, st, output_checkpoints=True)
        wg = gdr.scan_bwd(tx, tg, w[2], dout, w[1])
        for u, v in zip((o, f) + grads, w[:2] + wg):
            assert torch.equal(u, v)
    assert gdr.get_error() == 0


def test_wait_for_another_block_that_runs_out():
    """With the wait limit at 1 ns the blocks of a cluster give up waiting for one another: the calls end with
    GDR_DEVERR_TIMEOUT, and the next ones are right."""
    x, g, s0, r = draws(1, 1, 6000, 64, "f32", "f32", 570)
    tx, tg, st = dev(x, "f32"), dev(g, "f32"), dev(s0, "f32")
    want = gdr.scan_fwd(tx, tg, st, output_checkpoints=True)
    wg = gdr.scan_bwd(tx, tg, want[2], tx, st)
    gdr.set_wait_limit_ns(1)
    try:
        gdr.scan_fwd(tx, tg, st)
        assert gdr.get_error() == gdr.DEVERR_TIMEOUT
        gdr.scan_bwd(tx, tg, want[2], tx, st)
        assert gdr.get_error() == gdr.DEVERR_TIMEOUT
    finally:
        gdr.set_wait_limit_ns(0)
    for u, v in zip(gdr.scan_fwd(tx, tg, st) + gdr.scan_bwd(tx, tg, want[2], tx, st), want[:2] + (None,) + wg):
        assert v is None or torch.equal(u, v)
    assert gdr.get_error() == 0


def test_prepared_calls():
    x, g, s0, _ = draws(2, 2, 100, 64, "bf16", "f32", 560)
    tx, tg, st = dev(x, "bf16"), dev(g, "f32"), dev(s0, "f32")
    call = gdr.prepare_scan_fwd(tx, tg, st)
    out, fin, _ = call()
    want = gdr.scan_fwd(tx, tg, st)
    assert torch.equal(out, want[0]) and torch.equal(fin, want[1])
    tx.normal_()
    call()
    assert torch.equal(out, gdr.scan_fwd(tx, tg, st)[0])


@pytest.mark.parametrize("seed", range(40))
def test_random_cases(seed):
    r = np.random.default_rng(9000 + seed)
    dt, gt = TYPES[r.integers(len(TYPES))]
    B, N, D = int(r.integers(1, 5)), int(r.integers(1, 4)), int(np.exp(r.uniform(0, np.log(400))))
    S = int(np.exp(r.uniform(0, np.log(1200))))
    if r.random() < 0.5:
        D = max(8, D // 8 * 8)
    run_both(B, N, S, D, dt, gt, bool(r.integers(2)), bool(r.integers(2)), bool(r.integers(2)), 9100 + seed,
             dfinal=bool(r.integers(2)))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_state_and_gradient_in_place_with_clusters(dt):
    """final_state over initial_state and dinitial_state over dfinal_state where several blocks share a sequence, with an
    empty sequence and one that ends inside a tile."""
    B, N, S, D = 3, 1, 5000, 64
    x, g, s0, r = draws(B, N, S, D, dt, "f32", 580)
    L = np.array([5000, 0, 3333], np.int32)
    tx, tg, st = spoil(dev(x, dt), L), spoil(dev(g, "f32"), L), dev(s0, "f32")
    df = dev(rnd(r.normal(size=(B, N, D)), "f32"), "f32")
    out, fin, ck = gdr.scan_fwd(tx, tg, st.clone(), dev_i32(L), output_checkpoints=True)
    dout = spoil(dev(rnd(r.normal(size=x.shape), dt), dt), L)
    want = gdr.scan_bwd(tx, tg, ck, dout, df.clone(), dev_i32(L))
    o, f, _ = gdr.scan_fwd(tx, tg, st, dev_i32(L), final_state=st)
    got = gdr.scan_bwd(tx, tg, ck, dout, df, dev_i32(L), dinitial_state=df)
    assert f is st and got[2] is df and gdr.get_error() == 0
    for u, v in zip((o, f) + got, (out, fin) + want):
        assert torch.equal(u, v)
    _, rf, _ = R.scan_fwd(x, g, s0, L)
    E, _ = scan_bounds(x, g, s0, L, False)
    check(fin, rf, E[:, :, -1], "f32", "final_state")


def test_offsets_past_32_bits():
    """A tensor of more than 2^32 elements: behind a forgetting gate the end equals a call on the end alone."""
    S, D, tail = 131200, 32768, 100
    x = torch.full((1, 1, S, D), 0.25, dtype=torch.bfloat16, device="cuda")
    x[:, :, -tail:].normal_()
    g = torch.full((1, 1, S, D), -0.5, dtype=torch.bfloat16, device="cuda")
    g[:, :, -tail] = float("-inf")
    out, fin, ck = gdr.scan_fwd(x, g, output_checkpoints=True)
    xs, gs = x[:, :, -tail:].contiguous(), g[:, :, -tail:].contiguous()
    o, f, _ = gdr.scan_fwd(xs, gs)
    ro, rf, _ = R.scan_fwd(host(xs[..., :64]), host(gs[..., :64]))
    E, _ = scan_bounds(host(xs[..., :64]), host(gs[..., :64]), None, [tail], False)
    check(out[:, :, -tail:, :64], ro, E[:, :, 1:], "bf16", "out")
    check(fin[..., :64], rf, E[:, :, -1], "f32", "final_state")
    # the tiles lie otherwise in the short call, so sums are grouped otherwise: half a bf16 step apart at most, twice
    assert (out[:, :, -tail:].float() - o.float()).abs().max() <= 2 ** -7 * o.float().abs().max()
    # a constant input settles at x / (1 - a)
    assert abs(float(out[0, 0, -tail - 1, -1]) - 0.25 / (1 - np.exp(-0.5))) < 2 ** -8
    del out, o
    dx, dg, di = gdr.scan_bwd(x, g, ck, x)
    assert gdr.get_error() == 0
    a = np.exp(-0.5)
    assert abs(float(dx[0, 0, S // 2, -1]) - 0.25 / (1 - a)) < 2 ** -8
    assert abs(float(di[0, 0, -1]) - 0.25 * a / (1 - a)) < 1e-5
    assert not torch.any(dg[0, 0, -tail])  # nothing passes a forgotten state


@pytest.mark.timeout(300)
def test_two_host_threads_on_streams_of_their_own():
    import threading
    x, g, s0, _ = draws(2, 2, 1500, 128, "bf16", "f32", 590)
    tx, tg, st = dev(x, "bf16"), dev(g, "f32"), dev(s0, "f32")
    want = gdr.scan_fwd(tx, tg, st, output_checkpoints=True)
    wg = gdr.scan_bwd(tx, tg, want[2], tx, st)
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(30):
                o = gdr.scan_fwd(tx, tg, st, output_checkpoints=True)
                b = gdr.scan_bwd(tx, tg, o[2], tx, st)
                if not all(torch.equal(u, v) for u, v in zip(o + b, want + wg)):
                    bad.append(1)

    ts = [threading.Thread(target=work) for _ in range(2)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not bad and gdr.get_error() == 0


def test_step_for_more_sequences_than_a_grid_dimension():
    B = 70001
    x = torch.randn(B, 1, 1, 4, device="cuda")
    g = -torch.rand(B, 1, 1, 4, device="cuda")
    pool = torch.randn(B + 1, 1, 4, device="cuda")
    want = torch.exp(g.double())[:, :, 0] * pool[1:].double() + x.double()[:, :, 0]
    idx = torch.arange(1, B + 1, device="cuda", dtype=torch.int32)
    out, _ = gdr.scan_step(x, g, pool, idx)
    # one exponential (4 u), a product and a sum: 6 u of |a h| + |x|
    tol = 6 * 2.0 ** -24 * (torch.exp(g.double())[:, :, 0] * 8 + x.double().abs()[:, :, 0])
    assert bool(((pool[1:].double() - want).abs() <= tol).all()) and torch.equal(out[:, :, 0], pool[1:])


@pytest.mark.parametrize("dt,gt", TYPES)
@pytest.mark.parametrize("S,per_token", [(1, False), (1, True), (4, False), (5, True), (8, True)])
@pytest.mark.parametrize("N,D", [(2, 128), (3, 5)])
def test_step(dt, gt, S, per_token, N, D):
    B, mix = 6, S % 2 == 0
    slots = B * S + 3
    x, g, _, r = draws(B, N, S, D, dt, gt, 600 + S + D)
    pool = rnd(r.normal(size=(slots, N, D)), "f32")
    order = r.permutation(slots)
    idx = order[:B * S].reshape(B, S) if per_token else np.repeat(order[:B, None], S, 1)
    L = np.array([S, 0, max(1, S - 1), S, 1, S], np.int32)
    A = np.array([1, 1, S, max(1, S // 2), 1, S], np.int32)
    if not per_token:
        A[5] = 0
    tp = dev(pool, "f32")
    out, p = gdr.scan_step(spoil(dev(x, dt), L), spoil(dev(g, gt), L), tp, dev_i32(idx.reshape(-1)), dev_i32(L),
                           dev_i32(A), mix=mix, per_token=per_token)
    assert p is tp and gdr.get_error() == 0
    ro, rp = R.scan_step(x, g, pool, idx, L, A, mix, per_token)
    start = pool[[idx[b, A[b] - 1 if per_token else 0] for b in range(B)]]
    E, _ = scan_bounds(x, g, start, L, mix)
    check(out, ro, E[:, :, 1:], dt, "out")
    bound = np.zeros_like(pool)
    for b in range(B):
        for t in range(int(L[b]) if per_token else min(int(A[b]), int(L[b]))):
            bound[idx[b, t]] = E[b, :, t + 1]
    check(tp, rp, bound, "f32", "pool")
    left = np.setdiff1d(np.arange(slots), idx.reshape(-1))
    assert np.array_equal(host(tp)[left], pool[left])


def test_step_chain_reproduces_the_scan():
    """Decoding token by token, eager and as a replayed graph, reproduces the prefill's state within its bound."""
    x, g, s0, _ = draws(3, 2, 40, 128, "bf16", "f32", 640)
    tx, tg = dev(x, "bf16"), dev(g, "f32")
    pool = torch.zeros(5, 2, 128, device="cuda")
    pool[[4, 0, 2]] = dev(s0, "f32")
    idx = dev_i32([4, 0, 2])
    cx, cg = tx[:, :, :1].contiguous(), tg[:, :, :1].contiguous()
    gdr.scan_step(cx, cg, pool.clone(), idx)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = gdr.scan_step(cx, cg, pool, idx)
    outs = []
    for t in range(40):
        cx.copy_(tx[:, :, t:t + 1])
        cg.copy_(tg[:, :, t:t + 1])
        graph.replay()
        outs.append(out.clone())
    ro, rf, _ = R.scan_fwd(x, g, s0)
    E, _ = scan_bounds(x, g, s0, [40] * 3, False)
    check(torch.cat(outs, 2), ro, E[:, :, 1:], "bf16", "out")
    check(pool[[4, 0, 2]], rf, E[:, :, -1], "f32", "state")
    assert not torch.any(pool[[1, 3]])


def test_step_bad_slots_lengths_and_counts_are_skipped_and_flagged():
    x, g, _, r = draws(4, 1, 2, 12, "f32", "f32", 650)
    pool = torch.randn(6, 1, 12, device="cuda")
    tx, tg = dev(x, "f32"), dev(g, "f32")
    for idx, L, A, per_token, err in (
            ([0, 0, 6, 6, 2, 2, 3, 3], None, None, False, gdr.DEVERR_SLOT_INDEX),
            ([0, 0, 1, -1, 2, 2, 3, 3], None, None, False, gdr.DEVERR_SLOT_INDEX),
            ([0, 0, 1, 1, 2, 2, 3, 3], [2, 3, 2, 2], None, False, gdr.DEVERR_LENGTH),
            ([0, 0, 1, 4, 2, 2, 3, 3], None, [1, 0, 1, 1], True, gdr.DEVERR_LENGTH),
            ([0, 0, 1, 4, 2, 2, 3, 3], None, [1, 3, 1, 1], True, gdr.DEVERR_LENGTH)):
        p = pool.clone()
        out, _ = gdr.scan_step(tx, tg, p, dev_i32(idx), dev_i32(L), dev_i32(A), per_token=per_token)
        assert gdr.get_error() == err
        assert not torch.any(out[1]) and bool(torch.any(out[0])) and bool(torch.any(out[3]))
        assert torch.equal(p[[1, 4, 5]], pool[[1, 4, 5]]) and not torch.equal(p[0], pool[0])


def test_checked_mode(monkeypatch):
    monkeypatch.setenv("GDR_CHECKS", "1")
    e = torch.zeros(2, 1, 2, 4, device="cuda")
    pool = torch.zeros(4, 1, 4, device="cuda")
    gdr.scan_step(e, e, pool, dev_i32([0, 0, 1, 1]))
    with pytest.raises(ValueError):
        gdr.scan_step(e, e, pool, dev_i32([0, 0, 0, 0]))  # two sequences, one slot
    with pytest.raises(ValueError):
        gdr.scan_fwd(e, e, None, dev_i32([3, 0]))
    assert gdr.get_error() == 0


def test_binding_refusals():
    e = torch.zeros(2, 1, 6, 4, device="cuda")
    h = e.to(torch.bfloat16)
    with pytest.raises(RuntimeError):
        gdr.scan_fwd(e, h)  # a gate of fewer bits than the input
    with pytest.raises(RuntimeError):
        gdr.scan_fwd(h, e.half())
    with pytest.raises(ValueError):
        gdr.scan_fwd(e, e[:, :, :5])
    with pytest.raises(RuntimeError):
        gdr.scan_fwd(e.transpose(2, 3), e.transpose(2, 3))  # not dense
    with pytest.raises(RuntimeError):
        gdr.scan_fwd(h, h, torch.zeros(2, 1, 4, device="cuda", dtype=torch.bfloat16))  # the state is fp32
    with pytest.raises(ValueError):
        gdr.scan_fwd(e, e.clone(), out=e)  # in place
    with pytest.raises(ValueError):
        gdr.scan_bwd(e, e, torch.zeros(2, 1, 2, 4, device="cuda"), e)  # one checkpoint for each 64 tokens
    with pytest.raises(ValueError):
        gdr.scan_step(torch.zeros(1, 1, 9, 4, device="cuda"), torch.zeros(1, 1, 9, 4, device="cuda"),
                      torch.zeros(2, 1, 4, device="cuda"), torch.zeros(9, device="cuda", dtype=torch.int32))
    with pytest.raises(ValueError):
        gdr.scan_step(e, e, torch.zeros(2, 1, 4, device="cuda"), torch.zeros(3, device="cuda", dtype=torch.int32))
    assert gdr.get_error() == 0
