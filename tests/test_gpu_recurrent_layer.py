"""The operators together, as a recurrent layer uses them: conv1d, gated linear recurrence and output gate; its training
step, and its serving with prefix sharing, beam reordering, compaction and freeing of slots."""
import numpy as np
import pytest
import torch

import gated_deltanet_gdr_b200 as gdr
import oracle
from oracle import recurrence as R
from tests._bounds import check
from tests._helpers import dev, dev_i32, host, rnd

pytestmark = pytest.mark.gpu

N, D, K = 2, 64, 4
C = 3 * N * D


class Layer:
    """h = scan(v, -softplus(k)), y = h * q, with q, k, v = conv1d(x); the elementwise parts are torch's"""

    def __init__(self, seed):
        r = np.random.default_rng(seed)
        self.w, self.b = rnd(0.5 * r.normal(size=(C, K)), "f32"), rnd(0.1 * r.normal(size=C), "f32")
        self.tw, self.tb = dev(self.w, "f32"), dev(self.b, "f32")

    def forward(self, x, conv, h0, lens=None):
        q, k, v, nc = gdr.conv1d(x, self.tw, self.tb, conv, lens, Nk=N, Nv=N, Dk=D, Dv=D)
        g = -torch.nn.functional.softplus(k)
        out, fin, ck = gdr.scan_fwd(v, g, h0, lens, output_checkpoints=True)
        return out * q, (q, k, v, g, out, nc, fin, ck)

    def exact(self, x, conv, h0, lens=None):
        """the same in fp64 numpy"""
        y, nc = oracle.causal_conv1d(x, self.w, self.b, conv, lens)
        B, S, _ = x.shape
        q, k, v = (y[:, :, i * N * D:(i + 1) * N * D].reshape(B, S, N, D).transpose(0, 2, 1, 3) for i in range(3))
        out, fin, _ = R.scan_fwd(v, -np.logaddexp(0, k), h0, lens)
        return out * q, nc, fin


def test_training_step_against_differences():
    """Gradients of the whole layer against central differences of its fp64 form.  The step 1e-5 leaves e^2 |f'''| / 6 <
    1e-8 and rounds 2^-53 |loss| / e < 1e-8; the fp32 pass loses a few hundred roundings of 2^-24 in sums of a few
    hundred terms: 1e-4 of the gradient's size holds both with a margin."""
    r = np.random.default_rng(0)
    layer = Layer(1)
    B, S = 2, 70
    lens = np.array([70, 41], np.int32)
    x, conv, h0 = (rnd(r.normal(size=s), "f32") for s in ((B, S, C), (B, C, K), (B, N, D)))
    dy, dfin = rnd(r.normal(size=(B, N, S, D)), "f32"), rnd(r.normal(size=(B, N, D)), "f32")
    tx, tc, th, tl = dev(x, "f32"), dev(conv, "f32"), dev(h0, "f32"), dev_i32(lens)
    y, (q, k, v, g, out, nc, fin, ck) = layer.forward(tx, tc, th, tl)
    ey, _, ef = layer.exact(x, conv, h0, lens)
    assert np.abs(host(y) - ey).max() < 1e-4 and np.abs(host(fin) - ef).max() < 1e-4
    tdy = dev(dy, "f32")
    dout, dq = tdy * q, tdy * out
    dv, dg, dh0 = gdr.scan_bwd(v, g, ck, dout, dev(dfin, "f32"), tl)
    dk = -dg * torch.sigmoid(k)
    dx, dw, db, dconv = gdr.conv1d_bwd(tx, layer.tw, dq, dk, dv, layer.tb, tc, tl)
    assert gdr.get_error() == 0

    def loss(x, w, b, conv, h0):
        l = Layer.__new__(Layer)
        l.w, l.b = w, b
        y, _, f = l.exact(x, conv, h0, lens)
        return (y * dy).sum() + (f * dfin).sum()

    base = [x, layer.w, layer.b, conv, h0]
    e = 1e-5
    for i, got in enumerate((dx, dw, db, dconv, dh0)):
        got = host(got)
        scale = np.abs(got).max()
        for at in [tuple(r.integers(0, n) for n in got.shape) for _ in range(6)]:
            hi, lo = [a.copy() for a in base], [a.copy() for a in base]
            hi[i][at] += e
            lo[i][at] -= e
            num = (loss(*hi) - loss(*lo)) / (2 * e)
            assert abs(num - got[at]) <= 1e-4 * max(scale, 1.0), (i, at, num, got[at])


def test_serving_with_shared_prefixes_beams_and_compaction():
    """A prompt is prefilled into one slot and copied to four beams; beams are stepped, reordered and stepped again; the
    pool is compacted, stepped once more, and freed.  Every beam's outputs are those of its whole history in fp64."""
    r = np.random.default_rng(3)
    layer = Layer(4)
    slots, P, beams = 12, 37, 4
    prompt = rnd(r.normal(size=(1, P, C)), "f32")
    pool, convs = torch.zeros(slots, N, D, device="cuda"), torch.zeros(slots, C, K, device="cuda")
    live = torch.zeros(slots, dtype=torch.int32, device="cuda")
    _, st = layer.forward(dev(prompt, "f32"), None, None)
    pool[9], convs[9] = st[6][0], st[5][0]
    table = dev_i32([9, 3, 11, 6])
    live[table.long()] = 1
    gdr.slot_copy([pool, convs], dev_i32([9] * 3 + [-1]), dev_i32([3, 11, 6, -1]))
    history = [prompt[0]] * beams

    def step(tokens):
        """one token (beams, C) for every beam; checks the outputs against the whole histories"""
        nonlocal history
        history = [np.concatenate([h, t[None]]) for h, t in zip(history, tokens)]
        at = table.long()
        q, k, v, nc = gdr.conv1d(dev(tokens[:, None], "f32"), layer.tw, layer.tb, convs[at].contiguous(), None, Nk=N, Nv=N,
                                 Dk=D, Dv=D)
        convs[at] = nc
        h, _ = gdr.scan_step(v, -torch.nn.functional.softplus(k), pool, table)
        got = host(h * q)[:, :, 0]
        for i in range(beams):
            y, _, _ = layer.exact(history[i][None], None, None)
            # fp32 over a few dozen tokens with values of a few: a few hundred roundings of 2^-24
            assert np.abs(got[i] - y[0, :, -1]).max() < 1e-4, i

    for parents in ([0, 0, 2, 0], [3, 3, 1, 1], [2, 2, 2, 2]):
        step(rnd(r.normal(size=(beams, C)), "f32"))
        new = gdr.slot_fork([pool, convs], table, dev_i32(parents))
        assert sorted(new.tolist()) == sorted(table.tolist())
        table = new
        history = [history[p] for p in parents]
    where, n = gdr.slot_compact([pool, convs], live)
    assert int(n) == beams
    table = where[table.long()].contiguous()
    assert sorted(table.tolist()) == [0, 1, 2, 3]
    step(rnd(r.normal(size=(beams, C)), "f32"))
    live = (torch.arange(slots, device="cuda") < n).int()
    gdr.slot_free([pool, convs], table, live)
    assert not torch.any(pool[:beams]) and not torch.any(convs[:beams]) and not torch.any(live)
    assert gdr.get_error() == 0


def test_the_rules_own_pool_is_forked_and_compacted():
    """The matrix states of recurrent_step live in such a pool too: forked rows decode as their parents would."""
    torch.manual_seed(0)
    Nk, Nv, Dh, slots = 2, 4, 128, 10
    pool = (0.05 * torch.randn(slots, Nv, Dh, Dh, device="cuda")).to(torch.bfloat16)
    ref = pool.clone()
    table = dev_i32([7, 2, 9])
    new = gdr.slot_fork(pool, table, dev_i32([1, 1, 1]))
    q, k = (torch.randn(3, Nk, 1, Dh, device="cuda").to(torch.bfloat16) for _ in range(2))
    v, b = torch.randn(3, Nv, 1, Dh, device="cuda").to(torch.bfloat16), torch.rand(3, Nv, 1, device="cuda").to(torch.bfloat16)
    pro, ones = gdr.Prologue(l2norm_qk=True, eps=1e-6, beta_logits=False), dev_i32([1, 1, 1])
    out, _ = gdr.recurrent_step(q, k, v, b, None, None, pool, new, ones, scale=Dh ** -0.5, prologue=pro)
    for i in range(3):
        one = ref[2:3].clone()
        o, _ = gdr.recurrent_step(q[i:i + 1].clone(), k[i:i + 1].clone(), v[i:i + 1].clone(),
                                  b[i:i + 1].clone(), None, None, one, dev_i32([0]), dev_i32([1]), scale=Dh ** -0.5,
                                  prologue=pro)
        assert torch.equal(o[0], out[i]) and torch.equal(one[0], pool[int(new[i])])
    live = torch.zeros(slots, dtype=torch.int32, device="cuda")
    live[new.long()] = 1
    before = pool.clone()
    where, n = gdr.slot_compact(pool, live)
    assert torch.equal(pool[where[new.long()].long()], before[new.long()]) and int(n) == 3
    assert gdr.get_error() == 0
