"""Copying, forking, compacting and freeing state slots on the GPU: bit for bit the moves of the definition."""
import numpy as np
import pytest
import torch

import gated_deltanet_gdr_b200 as gdr
from oracle import recurrence as R
from tests._helpers import dev_i32

pytestmark = pytest.mark.gpu

# shapes of one slot and types: matrix states, conv windows, odd sizes down to single bytes, several pieces and a rest
POOLS = [((2, 32, 32), torch.bfloat16), ((48, 4), torch.bfloat16), ((2, 33), torch.float32), ((7,), torch.bfloat16),
         ((1,), torch.uint8), ((5, 3), torch.uint8), ((41, 1001), torch.uint8), ((4, 64, 64), torch.float32),
         ((20489,), torch.float32), ((3,), torch.float64)]


def make(slots, which=None, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    res = []
    for shape, dt in (POOLS if which is None else [POOLS[i] for i in which]):
        n = int(np.prod(shape)) * dt.itemsize
        raw = torch.randint(0, 256, (slots, n), generator=g, device="cuda", dtype=torch.uint8)
        res.append(raw.view(dt).reshape((slots,) + shape))
    return res


def raw(p):
    return p.contiguous().view(torch.uint8).reshape(p.shape[0], -1).cpu().numpy()


def same(pools, want):
    for i, (p, w) in enumerate(zip(pools, want)):
        assert np.array_equal(raw(p), w), i


@pytest.mark.parametrize("slots,n,pad", [(2, 1, 0), (9, 4, 3), (40, 20, 0), (300, 200, 50)])
def test_copy(slots, n, pad):
    pools = make(slots, seed=slots)
    r = np.random.default_rng(slots)
    order = r.permutation(slots)
    dst = np.concatenate([order[:n], [-1] * pad]).astype(np.int32)
    src = np.concatenate([order[n + r.integers(0, slots - n, n)], r.integers(-1, slots, pad)]).astype(np.int32)
    want, bad = R.slot_copy([raw(p) for p in pools], src, dst)
    assert not bad
    assert gdr.slot_copy(pools, dev_i32(src), dev_i32(dst)) is pools
    same(pools, want)
    assert gdr.get_error() == 0


@pytest.mark.parametrize("src,dst", [([1, 2], [2, 3]), ([0, 1], [4, 4]), ([0, 6], [1, 2]), ([0, 1], [-2, 2]),
                                     ([0, 3, 1], [3, 3, 1]), ([0, 1], [1, 0]), ([3, 5, 5], [4, 4, 3]),
                                     ([2 ** 30, 1], [0, 2]), ([-5, 1], [-1, 2])])
def test_copy_collisions_and_bad_slots_are_skipped_and_flagged(src, dst):
    pools = make(6, [0, 2, 6], seed=2)
    want, bad = R.slot_copy([raw(p) for p in pools], src, dst)
    gdr.slot_copy(pools, dev_i32(src), dev_i32(dst))
    same(pools, want)
    assert gdr.get_error() == (gdr.DEVERR_SLOT_INDEX if bad else 0)


@pytest.mark.parametrize("n,slots", [(1, 1), (2, 5), (31, 31), (64, 80), (1000, 1003)])
@pytest.mark.parametrize("kind", ["random", "one", "self", "cycle", "ends"])
def test_fork(n, slots, kind):
    which = None if slots < 100 else [1, 2, 3, 5]
    pools = make(slots, which, seed=n)
    r = np.random.default_rng(n)
    table = r.permutation(slots)[:n].astype(np.int32)
    parents = {"random": r.integers(0, n, n), "one": np.full(n, n // 2), "self": np.arange(n),
               "cycle": (np.arange(n) + 1) % n, "ends": np.where(r.random(n) < 0.4, -1, r.integers(0, n, n))}[kind]
    parents = parents.astype(np.int32)
    want, new, bad = R.slot_fork([raw(p) for p in pools], table, parents)
    assert not bad
    got = gdr.slot_fork(pools, dev_i32(table), dev_i32(parents))
    assert np.array_equal(got.cpu().numpy(), new)
    same(pools, want)
    assert gdr.get_error() == 0


@pytest.mark.parametrize("table,parents", [([0, 1, 2, 3], [0, 0, 9, -7]), ([0, 1, 9, 3], [0, 0, 1, 1]),
                                           ([0, 1, -1, 3], [2, 2, 2, 0]), ([0, 1, 1, 3], [0, 0, 3, 3]),
                                           ([2, 2, 2, 2], [1, 1, 1, 1])])
def test_fork_bad_parents_and_slots_are_skipped_and_flagged(table, parents):
    pools = make(6, [0, 3], seed=3)
    want, new, bad = R.slot_fork([raw(p) for p in pools], table, parents)
    got = gdr.slot_fork(pools, dev_i32(table), dev_i32(parents))
    assert bad and gdr.get_error() == gdr.DEVERR_SLOT_INDEX
    assert np.array_equal(got.cpu().numpy(), new)
    same(pools, want)


@pytest.mark.parametrize("slots", [1, 2, 31, 32, 33, 64, 100, 257, 5000])
@pytest.mark.parametrize("share", [0.0, 0.1, 0.6, 1.0])
def test_compact(slots, share):
    which = [0, 2, 6] if slots <= 257 else [1, 5]
    pools = make(slots, which, seed=slots)
    r = np.random.default_rng(slots)
    live = (r.random(slots) < share).astype(np.int32) * r.integers(1, 4, slots).astype(np.int32)
    want, new, n = R.slot_compact([raw(p) for p in pools], live)
    got, count = gdr.slot_compact(pools, dev_i32(live))
    assert int(count) == n and np.array_equal(got.cpu().numpy(), new)
    same(pools, want)
    # compacting again, with the places that are taken now, moves nothing
    again, _ = gdr.slot_compact(pools, (torch.arange(slots, device="cuda") < n).int())
    same(pools, want)


def test_compact_keeps_the_live_slots_at_the_front():
    for live, moved in (([1, 1, 1, 0, 0], {}), ([0, 0, 0, 1, 1], {3: 0, 4: 1}), ([0] * 5, {}), ([1] * 5, {})):
        pools = make(5, [3])
        _, new, _ = R.slot_compact([raw(p) for p in pools], live)
        got, _ = gdr.slot_compact(pools, dev_i32(live))
        assert np.array_equal(got.cpu().numpy(), new) and all(new[s] == d for s, d in moved.items())


@pytest.mark.parametrize("idx", [[3], [0, 5, 3], [2, 2, -1, 2], [-1, -1], [6, 1], [-2, 4]])
@pytest.mark.parametrize("with_live", [False, True])
def test_free(idx, with_live):
    pools = make(6, seed=9)
    live = np.ones(6, np.int32) if with_live else None
    want, lv, bad = R.slot_free([raw(p) for p in pools], idx, live)
    tl = dev_i32(live) if with_live else None
    gdr.slot_free(pools, dev_i32(idx), tl)
    same(pools, want)
    assert not with_live or np.array_equal(tl.cpu().numpy(), lv)
    assert gdr.get_error() == (gdr.DEVERR_SLOT_INDEX if bad else 0)


def test_slots_past_four_gigabytes():
    """Offsets beyond 32 bits: the last slots of a 6 GB pool."""
    slots = 6 * 1024
    pool = torch.zeros((slots, 1 << 18), dtype=torch.float32, device="cuda")
    pool[1].normal_()
    gdr.slot_copy(pool, dev_i32([1, 1]), dev_i32([slots - 1, 5000]))
    assert torch.equal(pool[slots - 1], pool[1]) and torch.equal(pool[5000], pool[1])
    live = torch.zeros(slots, dtype=torch.int32, device="cuda")
    live[slots - 1] = 1
    new, n = gdr.slot_compact([pool], live)
    assert int(n) == 1 and int(new[slots - 1]) == 0 and torch.equal(pool[0], pool[1])
    gdr.slot_free(pool, dev_i32([slots - 1]))
    assert not torch.any(pool[slots - 1]) and torch.equal(pool[5000], pool[1])
    assert gdr.get_error() == 0


def test_many_pools_many_moves_and_a_graph():
    pools = [torch.randn(50, 3 + i, device="cuda") for i in range(64)]
    keep = [p.clone() for p in pools]
    table, parents = dev_i32(np.arange(50)[::-1]), dev_i32(np.arange(50) // 2)
    new = torch.empty(50, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdr.slot_fork(pools, table, parents, new_slot_table=new)
    graph.replay()
    for p, k in zip(pools, keep):
        assert torch.equal(p[new.long()], k[table.long()[parents.long()]])
    parents.copy_(dev_i32(np.arange(50)))
    graph.replay()
    assert torch.equal(new, table)
    big = torch.arange(40000, device="cuda").reshape(-1, 1).repeat(1, 2)
    src, dst = torch.arange(0, 20000, device="cuda").int(), torch.arange(20000, 40000, device="cuda").int()
    gdr.slot_copy(big, src, dst)
    assert torch.equal(big[20000:], big[:20000])
    assert gdr.get_error() == 0


def test_refusals():
    p = torch.zeros(4, 8, device="cuda")
    i = dev_i32([0])
    with pytest.raises(ValueError):
        gdr.slot_copy([], i, i)
    with pytest.raises(ValueError):
        gdr.slot_copy([p, torch.zeros(5, 8, device="cuda")], i, i)
    with pytest.raises(ValueError):
        gdr.slot_copy([p] * 2, i, i)  # the same pool twice
    with pytest.raises(ValueError):
        gdr.slot_copy([torch.zeros(4, 1, device="cuda") for _ in range(65)], i, i)
    with pytest.raises(ValueError):
        gdr.slot_copy(p, i, dev_i32([1, 2]))
    with pytest.raises(RuntimeError):
        gdr.slot_copy(p, i, torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(RuntimeError):
        gdr.slot_copy(p.t(), i, i)
    t = dev_i32([0, 1])
    with pytest.raises(ValueError):
        gdr.slot_fork(p, t, t.clone(), new_slot_table=t)
    with pytest.raises(ValueError):
        gdr.slot_compact(p, dev_i32([1, 1, 1]))
    with pytest.raises(ValueError):
        gdr.slot_free(p, i, dev_i32([1, 1]))
    gdr.slot_copy(p, i[:0], i[:0])  # nothing to do
    gdr.slot_free(p, i[:0])
    gdr.slot_fork(p, i[:0], i[:0])
    assert gdr.get_error() == 0
