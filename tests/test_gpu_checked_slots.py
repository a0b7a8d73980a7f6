"""Checked mode (GDR_CHECKS=1) of the slot calls and of the conv1d: what a kernel would skip and flag is refused before the
launch, with nothing moved, and so is a slot that two rows of a fork share."""
import pytest
import torch

import gated_deltanet_gdr_b200 as gdr
from tests._helpers import dev_i32

pytestmark = pytest.mark.gpu


@pytest.fixture
def pools(monkeypatch):
    monkeypatch.setenv("GDR_CHECKS", "1")
    p = [torch.randn(6, 3, 5, device="cuda"), torch.randn(6, 7, device="cuda").half()]
    yield p
    assert gdr.get_error() == 0


def refused(pools, f, *args):
    before = [p.clone() for p in pools]
    with pytest.raises(ValueError):
        f(pools, *args)
    assert all(torch.equal(u, v) for u, v in zip(pools, before))


@pytest.mark.parametrize("src,dst", [([1, 2], [2, 3]), ([0, 1], [4, 4]), ([0, 6], [1, 2]), ([0, 1], [-2, 2]),
                                     ([0, 3, 1], [3, 2, 5]), ([0, 1], [1, 0]), ([2 ** 30, 1], [0, 2]), ([-5, 1], [3, 2])])
def test_copies_that_collide_or_are_out_of_range(pools, src, dst):
    refused(pools, gdr.slot_copy, dev_i32(src), dev_i32(dst))


@pytest.mark.parametrize("src,dst", [([], []), ([0, 0, 1], [3, 4, 5]), ([-1, 7, 2], [9, -1, 2]), ([2, 2, 2], [2, 3, 2])])
def test_copies_that_are_right(pools, src, dst):
    want = [p.clone() for p in pools]
    for s, d in zip(src, dst):
        if s != -1 and d != -1 and s != d:
            for w, p in zip(want, pools):
                w[d] = p[s]
    gdr.slot_copy(pools, dev_i32(src), dev_i32(dst))
    assert all(torch.equal(u, v) for u, v in zip(pools, want))


@pytest.mark.parametrize("table,parents", [([0, 1, 2], [0, 3, 1]), ([0, 1, 2], [-2, 0, 1]), ([0, 1, 1], [0, 0, 2]),
                                           ([0, 1, 1], [0, 1, 2]), ([0, 6, 2], [0, 0, 2]), ([-1, 1, 2], [0, 0, 2])])
def test_forks_with_bad_parents_or_slots(pools, table, parents):
    refused(pools, gdr.slot_fork, dev_i32(table), dev_i32(parents))


@pytest.mark.parametrize("table,parents", [([4, 1, 2], [0, 0, -1]), ([4, 1, 2], [2, 2, 2]), ([5, -1, -1], [0, -1, -1]),
                                           ([0, 1], [1, 0]), ([3], [-1])])
def test_forks_that_are_right(pools, table, parents, monkeypatch):
    other = [p.clone() for p in pools]
    now = gdr.slot_fork(pools, dev_i32(table), dev_i32(parents))
    monkeypatch.delenv("GDR_CHECKS")
    assert torch.equal(now, gdr.slot_fork(other, dev_i32(table), dev_i32(parents)))
    assert all(torch.equal(u, v) for u, v in zip(pools, other))


def test_freeing(pools):
    live = torch.ones(6, dtype=torch.int32, device="cuda")
    for idx in ([6], [0, -2], [1, 2 ** 30]):
        refused(pools, gdr.slot_free, dev_i32(idx), live)
    assert bool(live.all())
    gdr.slot_free(pools, dev_i32([3, -1, 3]), live)
    assert live.tolist() == [1, 1, 1, 0, 1, 1] and not any(bool(p[3].any()) for p in pools)


def test_compaction_has_nothing_to_refuse(pools):
    new, n = gdr.slot_compact(pools, dev_i32([0, 7, -3, 0, 1, 0]))
    assert new.tolist() == [-1, 1, 2, -1, 0, -1] and int(n) == 3


def test_the_lengths_of_the_conv(pools):
    x, w = torch.zeros(2, 4, 48, device="cuda"), torch.zeros(48, 4, device="cuda")
    heads = dict(Nk=1, Nv=1, Dk=16, Dv=16)
    d = torch.zeros(2, 1, 4, 16, device="cuda")
    gdr.conv1d(x, w, None, None, dev_i32([4, 0]), **heads)
    for bad in ([5, 0], [0, -1]):
        with pytest.raises(ValueError):
            gdr.conv1d(x, w, None, None, dev_i32(bad), **heads)
        with pytest.raises(ValueError):
            gdr.conv1d_bwd(x, w, d, d, d, None, None, dev_i32(bad))
