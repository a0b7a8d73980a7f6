"""numpy fp64 definitions of the gated linear recurrence, the conv1d's gradient and the state-slot operators.

Each is written out from its definition, token by token or move by move; the pins are in
``tests/test_oracle_recurrence.py``.  Test infrastructure only, like the rest of this package.
"""
from __future__ import annotations

import numpy as np

CHUNK = 64


def _terms(x, g, mix):
    a = np.exp(g)
    return a, (-np.expm1(g) * x if mix else x)


def scan_fwd(x, g, h0=None, lengths=None, mix=False):
    """(out, final, checkpoints): x, g (B, N, S, D); checkpoints (B, N, ceil(S / 64), D), NaN where none is defined."""
    B, N, S, D = x.shape
    lengths = np.full(B, S) if lengths is None else np.asarray(lengths)
    h = np.zeros((B, N, D)) if h0 is None else np.array(h0, np.float64)
    out = np.zeros((B, N, S, D))
    ck = np.full((B, N, -(-S // CHUNK), D), np.nan)
    for b in range(B):
        for t in range(int(lengths[b])):
            if t % CHUNK == 0:
                ck[b, :, t // CHUNK] = h[b]
            a, w = _terms(x[b, :, t], g[b, :, t], mix)
            h[b] = a * h[b] + w
            out[b, :, t] = h[b]
        if lengths[b] == 0 and S > 0:
            ck[b, :, 0] = h[b]
    return out, h, ck


def scan_bwd(x, g, h0, dout, dfinal=None, lengths=None, mix=False):
    """(dx, dg, dinitial) by the chain rule, last token first."""
    B, N, S, D = x.shape
    lengths = np.full(B, S) if lengths is None else np.asarray(lengths)
    mu = np.zeros((B, N, D)) if dfinal is None else np.array(dfinal, np.float64)
    dx, dg = np.zeros((B, N, S, D)), np.zeros((B, N, S, D))
    for b in range(B):
        h = np.zeros((N, D)) if h0 is None else np.array(h0[b], np.float64)
        before = []
        for t in range(int(lengths[b])):
            before.append(h)
            a, w = _terms(x[b, :, t], g[b, :, t], mix)
            h = a * h + w
        for t in reversed(range(int(lengths[b]))):
            lam = dout[b, :, t] + mu[b]  # d loss / d h_t
            a = np.exp(g[b, :, t])
            dx[b, :, t] = -np.expm1(g[b, :, t]) * lam if mix else lam
            dg[b, :, t] = lam * a * (before[t] - x[b, :, t] if mix else before[t])
            mu[b] = lam * a
    return dx, dg, mu


def scan_step(x, g, pool, indices, lengths=None, accepted=None, mix=False, per_token=False):
    """(out, pool after): pool (slots, N, D), indices (B * S)."""
    B, N, S, D = x.shape
    pool = np.array(pool, np.float64)
    idx = np.asarray(indices).reshape(B, S)
    out = np.zeros((B, N, S, D))
    for b in range(B):
        L = S if lengths is None else int(lengths[b])
        if L == 0:
            continue
        if per_token:
            start, keep = (1 if accepted is None else int(accepted[b])) - 1, L
        else:
            start, keep = 0, (L if accepted is None else min(int(accepted[b]), L))
        h = pool[idx[b, start]].copy()
        for t in range(L):
            a, w = _terms(x[b, :, t], g[b, :, t], mix)
            h = a * h + w
            out[b, :, t] = h
            if t < keep:
                pool[idx[b, t]] = h
    return out, pool


def conv1d_bwd(x, w, bias, state, lengths, dy, dstate_out=None):
    """(dx, dw, dbias, dstate): x, dy (B, S, C), w (C, K), state and dstate_out (B, C, K) or None."""
    B, S, C = x.shape
    K = w.shape[1]
    lengths = np.full(B, S) if lengths is None else np.asarray(lengths)
    dx, dw, db, ds = np.zeros((B, S, C)), np.zeros((C, K)), np.zeros(C), np.zeros((B, C, K))
    for b in range(B):
        L = int(lengths[b])
        hist = np.zeros((K + L, C))  # the state, then the valid inputs
        if state is not None:
            hist[:K] = state[b].T
        hist[K:] = x[b, :L]
        dhist = np.zeros((K + L, C))
        for t in range(L):
            pre = (w.T * hist[t + 1:t + 1 + K]).sum(0) + (0.0 if bias is None else bias)
            s = 1.0 / (1.0 + np.exp(-pre))
            d = dy[b, t] * (s + pre * s * (1.0 - s))
            dhist[t + 1:t + 1 + K] += w.T * d
            dw += (hist[t + 1:t + 1 + K] * d).T
            db += d
        if dstate_out is not None:
            dhist[L:] += dstate_out[b].T
        ds[b] = dhist[:K].T
        dx[b, :L] = dhist[K:]
    return dx, dw, db, ds


# ---- slots: pools are lists of numpy arrays (slots, ...); (result, whether an error is flagged) ---------------------


def slot_copy(pools, src, dst):
    slots = pools[0].shape[0]
    moves, bad = [], False
    for i, (s, d) in enumerate(zip(src, dst)):
        if s == -1 or d == -1 or s == d:
            continue
        if not (0 <= s < slots and 0 <= d < slots):
            bad = True
            continue
        moves.append((i, int(s), int(d)))
    keep = []
    for i, s, d in moves:
        if any(j != i and (d == sj or (d == dj and j < i)) for j, sj, dj in moves):
            bad = True
        else:
            keep.append((s, d))
    res = [p.copy() for p in pools]
    for s, d in keep:
        for p, r in zip(pools, res):
            r[d] = p[s]
    return res, bad


def slot_fork(pools, table, parents):
    """(pools, new table, flagged)"""
    slots, n = pools[0].shape[0], len(table)
    bad = any(not -1 <= r < n for r in parents)
    kids = [[i for i in range(n) if parents[i] == r] for r in range(n)]
    new = [None] * n
    for r in range(n):
        if kids[r]:
            new[kids[r][0]] = table[r]
    left = [r for r in range(n) if not kids[r]]
    res = [p.copy() for p in pools]
    for i in range(n):
        if new[i] is not None:
            continue
        row = left.pop(0)
        new[i] = table[row]
        if 0 <= parents[i] < n:
            s, d = table[parents[i]], table[row]
            if not (0 <= s < slots and 0 <= d < slots) or sum(1 for v in table if v == d) > 1:
                bad = True
                continue
            for p, r in zip(pools, res):
                r[d] = p[s]
    return res, np.array(new, np.int32), bad


def slot_compact(pools, live):
    """(pools, new_slot, n_live)"""
    used = [i for i, v in enumerate(live) if v]
    n = len(used)
    holes = [i for i in range(n) if not live[i]]
    new = np.full(len(live), -1, np.int32)
    res = [p.copy() for p in pools]
    for s in used:
        new[s] = s if s < n else holes.pop(0)
        for p, r in zip(pools, res):
            r[new[s]] = p[s]
    return res, new, n


def slot_free(pools, idx, live=None):
    """(pools, live, flagged)"""
    slots = pools[0].shape[0]
    res = [p.copy() for p in pools]
    live = None if live is None else live.copy()
    bad = False
    for i in idx:
        if 0 <= i < slots:
            for r in res:
                r[i] = 0
            if live is not None:
                live[i] = 0
        elif i != -1:
            bad = True
    return res, live, bad
