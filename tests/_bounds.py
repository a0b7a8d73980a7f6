"""Error bounds of the fp32 kernels, from the arithmetic they may do, evaluated in fp64 next to the exact values.

u = 2^-24 is the largest relative error of one fp32 rounding.  What each call may lose:

  recurrence   every state is a sum over s of (product of the decays after s) * b_s, however the scan groups it.  A factor
               e^g costs 4 u (CUDA's expf: 2 ulp) and one product 1 u, an addition 1 u, and regrouping at most doubles
               the products and additions of a token: 4 + 2 + 2 = 8 u of the absolute sum H for every token on the way.
               A write of the mixing form has (1 - a) x: 1 - a loses (4 a + 1) u / (1 - a) <= 19 u where |g| >= 1/4
               (a <= 0.78), and the series below that loses under 8 u; the product adds 1 u: 20 u of |b|.
               So E_t = a_t E_{t-1} + u (8 H_t + 20 |b_t|), with H the same recurrence of |b|.
  its gradient mu obeys the same recurrence backwards with dout for b: the same bound without the 20.  dx adds 20 u of
               its value in the mixing form; dg = mu (h - x) adds |mu| E + |h - x| E_mu and 3 u of the absolute product.
  outputs      one rounding to the output's type: eps / 2 of the value, plus half the smallest fp16 step (2^-25), and a
               fp32 product below 2^-126 may be lost.
"""
import numpy as np
import torch

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -25}


def _run(a, b, first):
    """the recurrence h = a h + b along axis 2"""
    out = np.empty_like(b)
    h = first
    for t in range(b.shape[2]):
        h = a[:, :, t] * h + b[:, :, t]
        out[:, :, t] = h
    return out


def scan_bounds(x, g, h0, lengths, mix):
    """(E, H): error bound and absolute sum of every state (B, N, S + 1, D), entry t the state before token t"""
    B, N, S, D = x.shape
    on = (np.arange(S)[None, :] < np.asarray(lengths)[:, None])[:, None, :, None]
    a = np.where(on, np.exp(np.where(on, g, 0.0)), 1.0)
    b = np.where(on, np.abs(np.where(on, (1 - a) if mix else 1.0, 0.0) * np.where(on, x, 0.0)), 0.0)
    first = np.zeros((B, N, D)) if h0 is None else np.abs(h0)
    H = _run(a, b, first)
    E = _run(a, np.where(on, U * (8 * H + (20 if mix else 0) * b), 0.0), np.zeros((B, N, D)))
    cat = lambda f, r: np.concatenate([f[:, :, None], r], 2)
    return cat(np.zeros((B, N, D)), E), cat(first, H)


def bwd_bounds(x, g, h0, lengths, mix, dout, dfinal, E, H, h):
    """bounds of dx, dg, dinitial before their rounding; h the exact states (B, N, S + 1, D)"""
    B, N, S, D = x.shape
    on = (np.arange(S)[None, :] < np.asarray(lengths)[:, None])[:, None, :, None]
    clean = lambda v: np.where(on, np.where(on, v, 0.0), 0.0)
    a = np.where(on, np.exp(np.where(on, g, 0.0)), 1.0)
    mu = np.zeros((B, N, D)) if dfinal is None else np.abs(dfinal)
    e = np.zeros((B, N, D))
    bx, bg = np.zeros((B, N, S, D)), np.zeros((B, N, S, D))
    xa, da = np.abs(clean(x)), np.abs(clean(dout))
    for t in reversed(range(S)):
        lam, el = da[:, :, t] + mu, e + U * (da[:, :, t] + mu)
        w = (1 - a[:, :, t]) if mix else np.ones_like(lam)
        bx[:, :, t] = w * el + (20 * U * w * lam if mix else 0.0)
        ok = on[:, :, t]
        mu_n = np.where(ok, a[:, :, t] * lam, mu)
        e = np.where(ok, a[:, :, t] * el + 8 * U * mu_n, e)
        mu = mu_n
        diff = H[:, :, t] + (xa[:, :, t] if mix else 0.0)
        bg[:, :, t] = mu * (E[:, :, t] + 3 * U * diff) + diff * e
    return clean(bx), clean(bg), e


def check(got, want, bound, dt, what):
    """got (torch or numpy) against want within bound plus one rounding to dt"""
    got = got.detach().double().cpu().numpy() if isinstance(got, torch.Tensor) else np.asarray(got, np.float64)
    tol = np.broadcast_to(bound + HALF[dt] * (np.abs(want) + bound) + TINY[dt], want.shape)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.size, tuple(np.argwhere(bad)[0]), float(got[bad][0]),
                           float(want[bad][0]), float(tol[bad][0]))
