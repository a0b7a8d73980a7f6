"""The workloads of the gated linear recurrence, the state-slot operators and the conv1d backward.

Every case names one call of the library (``gdr.scan_fwd``, ``scan_bwd``, ``scan_step``, ``slot_copy``, ``slot_fork``,
``slot_compact``, ``slot_free``, ``conv1d_bwd``).  ``run`` computes it either in a plain form made of elementary torch
operations in fp32 (``own`` false) or by the library's call (``own`` true), on the same inputs.  ``exact`` evaluates
the definitions token by token in fp64.

Layouts are the library's: activations (B, N, S, D), recurrent states (B, N, D) or pools (slots, ...), conv inputs
(B, S, C) channels last with C = 2 * Nk * Dk + Nv * Dv.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CHUNK = 64  # tokens between two checkpointed states of the recurrence


def _bytes(name):
    return DT[name].itemsize


# ---- the cases ---------------------------------------------------------------------------------------------


def listed():
    return [
        # prefill of the recurrence at the layout of the repository's prefill workload, gates in fp32
        {"name": "scan_fwd_prefill", "op": "scan_fwd", "B": 4, "N": 32, "S": 4096, "D": 128, "dtype": "bf16", "gate": "f32",
         "mix": False, "h0": True, "ragged": False},
        # one long sequence with channels last: few chains, so the work has to be split over time
        {"name": "scan_fwd_one_long", "op": "scan_fwd", "B": 1, "N": 1, "S": 32769, "D": 640, "dtype": "f16", "gate": "f16",
         "mix": True, "h0": False, "ragged": False},
        # the training step's gradient at the same layout
        {"name": "scan_bwd_train", "op": "scan_bwd", "B": 4, "N": 32, "S": 4096, "D": 128, "dtype": "bf16", "gate": "f32",
         "mix": False, "h0": True, "ragged": False},
        # the gradient of a padded fp32 batch with odd sizes and one empty sequence
        {"name": "scan_bwd_padded", "op": "scan_bwd", "B": 7, "N": 5, "S": 777, "D": 100, "dtype": "f32", "gate": "f32",
         "mix": True, "h0": True, "ragged": True},
        # one token for each of 64 sequences: the latency of a decode step
        {"name": "scan_step_decode", "op": "scan_step", "B": 64, "N": 32, "S": 1, "D": 128, "dtype": "bf16", "gate": "f32",
         "mix": False, "per_token": False, "slots": 128},
        # drafted tokens with a slot of their own each, for a large batch
        {"name": "scan_step_drafts", "op": "scan_step", "B": 256, "N": 32, "S": 4, "D": 128, "dtype": "f16", "gate": "f16",
         "mix": True, "per_token": True, "slots": 1100},
        # prompts' states copied to new sequences: the matrix state and the conv window of the bench's decode layout
        {"name": "slot_copy_prefixes", "op": "slot_copy", "slots": 192, "n": 96, "Nv": 32, "Dk": 128, "Dv": 128, "C": 8192,
         "K": 4, "state": "bf16", "pad": 8},
        # beam search reorders 64 beams
        {"name": "slot_fork_beams", "op": "slot_fork", "slots": 80, "n": 64, "Nv": 16, "Dk": 128, "Dv": 128, "C": 4096, "K": 4,
         "state": "f32", "pad": 0},
        # a pool of 512 slots, 60 % of them in use, is closed up
        {"name": "slot_compact_pool", "op": "slot_compact", "slots": 512, "n": 307, "Nv": 32, "Dk": 128, "Dv": 128, "C": 8192,
         "K": 4, "state": "bf16", "pad": 0},
        # a few finished sequences give their slots back
        {"name": "slot_free_few", "op": "slot_free", "slots": 33, "n": 5, "Nv": 4, "Dk": 64, "Dv": 64, "C": 768, "K": 4,
         "state": "bf16", "pad": 3},
        # the conv's gradient at the repository's conv1d layout
        {"name": "conv1d_bwd_train", "op": "conv1d_bwd", "B": 4, "S": 4096, "Nk": 16, "Nv": 32, "Dk": 128, "Dv": 128, "K": 4,
         "dtype": "bf16", "bias": True, "state": True, "ragged": False},
        # a small padded batch with other head sizes and three taps
        {"name": "conv1d_bwd_padded", "op": "conv1d_bwd", "B": 3, "S": 515, "Nk": 2, "Nv": 4, "Dk": 64, "Dv": 32, "K": 3,
         "dtype": "f32", "bias": True, "state": True, "ragged": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_bwd", "scan_step", "slot_copy", "slot_fork", "slot_compact", "slot_free", "conv1d_bwd"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op in ("scan_fwd", "scan_bwd"):
        B, N, S = _log_int(rng, 1, 32), _log_int(rng, 1, 32), _log_int(rng, 1, 65536)
        D = rng.choice([1, 7, 33, 64, 96, 100, 128, 130, 256, 640, 1000, 2048, 4095, 4096])
        while B * N * S * D > 1 << 25:
            if S > 64 and rng.random() < 0.5:
                S = max(1, S // 2 - rng.randrange(2))
            elif B > 1:
                B = B // 2
            elif N > 1:
                N = N // 2
            else:
                S = max(1, S // 2)
        return {"op": op, "B": B, "N": N, "S": S, "D": D, "dtype": dtype, "gate": rng.choice([dtype, "f32"]),
                "mix": rng.random() < 0.5, "h0": rng.random() < 0.5, "ragged": rng.random() < 0.5}
    if op == "scan_step":
        B, S = _log_int(rng, 1, 512), rng.choice([1, 1, 1, 2, 4, 5, 8])
        per_token = S > 1 and rng.random() < 0.5
        return {"op": op, "B": B, "N": _log_int(rng, 1, 32), "S": S, "D": rng.choice([16, 33, 64, 100, 128, 256]), "dtype": dtype,
                "gate": rng.choice([dtype, "f32"]), "mix": rng.random() < 0.5, "per_token": per_token,
                "slots": B * (S if per_token else 1) + rng.randrange(1, 64)}
    if op == "conv1d_bwd":
        B, S, Nk = _log_int(rng, 1, 16), _log_int(rng, 1, 8192), rng.choice([1, 2, 4, 8])
        Nv, Dk, Dv = Nk * rng.choice([1, 2, 3]), rng.choice([16, 32, 64, 128]), rng.choice([16, 32, 64, 128])
        while B * S * (2 * Nk * Dk + Nv * Dv) > 1 << 25:
            S = max(1, S // 2 - rng.randrange(2))
        return {"op": op, "B": B, "S": S, "Nk": Nk, "Nv": Nv, "Dk": Dk, "Dv": Dv, "K": rng.choice([1, 2, 3, 4, 4, 5, 8]),
                "dtype": dtype, "bias": rng.random() < 0.5, "state": rng.random() < 0.5, "ragged": rng.random() < 0.5}
    slots, state = _log_int(rng, 2, 512), rng.choice(["f32", "bf16", "f16"])
    Nv, Dk, Dv = rng.choice([1, 4, 16, 32]), rng.choice([16, 64, 128]), rng.choice([16, 64, 128])
    while slots * Nv * Dk * Dv * _bytes(state) > 1 << 28:
        slots = max(2, slots // 2)
    n = rng.randrange(1, max(2, slots // 2 + 1)) if op in ("slot_copy", "slot_free") else rng.randrange(1, slots + 1)
    return {"op": op, "slots": slots, "n": n, "Nv": Nv, "Dk": Dk, "Dv": Dv, "C": 2 * Nv * Dk + Nv * Dv, "K": rng.choice([3, 4]),
            "state": state, "pad": rng.choice([0, 0, 1, 5]) if op in ("slot_copy", "slot_free") else 0}


# ---- the inputs ----------------------------------------------------------------------------------------------


def _lengths(B, S, ragged):
    """Valid tokens of each sequence: all of them, or spread evenly from 0 to S (a padded batch)."""
    if not ragged:
        return [S] * B
    return [S * b // (B - 1) for b in range(B)] if B > 1 else [max(1, S - S // 3)]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFF)


def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _log_decay(gen, shape, dtype):
    """-exp(A) softplus(a) with the rate exp(A) of each channel spread from 1/200 to 2: memories of one to hundreds of
    tokens, as trained gates have."""
    rate = torch.exp(torch.empty(shape[-1], device="cuda").uniform_(math.log(5e-3), math.log(2.0), generator=gen))
    raw = torch.randn(shape, generator=gen, device="cuda")
    return (-rate * torch.nn.functional.softplus(raw)).to(dtype)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen, op = _gen(seed), case["op"]
    st = {"case": case}
    if op in ("scan_fwd", "scan_bwd", "scan_step"):
        B, N, S, D = case["B"], case["N"], case["S"], case["D"]
        dt, gt = DT[case["dtype"]], DT[case["gate"]]
        st["x"] = _normal(gen, (B, N, S, D), dt)
        st["g"] = _log_decay(gen, (B, N, S, D), gt)
    if op in ("scan_fwd", "scan_bwd"):
        st["h0"] = _normal(gen, (B, N, D), torch.float32) if case["h0"] else None
        st["lens"] = _i32(_lengths(B, S, True)) if case["ragged"] else None
        if op == "scan_bwd":
            # what the forward pass left behind: the states before each chunk of 64 tokens
            h = _scan(st["x"], st["g"], st["h0"], st["lens"], case["mix"])[0]
            first = st["h0"] if st["h0"] is not None else torch.zeros((B, N, D), device="cuda")
            st["checkpoints"] = torch.cat([first[:, :, None], h[:, :, CHUNK - 1:S - 1:CHUNK]], dim=2).contiguous()
            st["dout"] = _normal(gen, (B, N, S, D), dt)
            st["dfinal"] = _normal(gen, (B, N, D), torch.float32)
    elif op == "scan_step":
        slots = case["slots"]
        st["pool"] = _normal(gen, (slots, N, D), torch.float32)
        order = torch.randperm(slots, generator=gen, device="cuda").to(torch.int32)
        if case["per_token"]:  # every drafted token has a slot, the last call accepted some of its tokens
            st["idx"] = order[:B * S].contiguous()
            st["accepted"] = torch.randint(1, S + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
            st["lens"] = torch.randint(1, S + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        else:
            st["idx"] = order[:B].repeat_interleave(S).contiguous()
            st["accepted"], st["lens"] = None, None
    elif op == "conv1d_bwd":
        B, S, K, dt = case["B"], case["S"], case["K"], DT[case["dtype"]]
        Nk, Nv, Dk, Dv = case["Nk"], case["Nv"], case["Dk"], case["Dv"]
        C = 2 * Nk * Dk + Nv * Dv
        st["x"] = _normal(gen, (B, S, C), dt)
        st["weight"] = _normal(gen, (C, K), dt, 0.5 / math.sqrt(K))
        st["bias"] = _normal(gen, (C,), dt, 0.1) if case["bias"] else None
        st["conv_state"] = _normal(gen, (B, C, K), dt) if case["state"] else None
        st["dstate_out"] = _normal(gen, (B, C, K), dt) if case["state"] else None
        st["lens"] = _i32(_lengths(B, S, True)) if case["ragged"] else None
        st["dq"] = _normal(gen, (B, Nk, S, Dk), dt)
        st["dk"] = _normal(gen, (B, Nk, S, Dk), dt)
        st["dv"] = _normal(gen, (B, Nv, S, Dv), dt)
    else:
        slots, n, dt = case["slots"], case["n"], DT[case["state"]]
        st["pools"] = [_normal(gen, (slots, case["Nv"], case["Dk"], case["Dv"]), dt),
                       _normal(gen, (slots, case["C"], case["K"]), dt)]
        order = torch.randperm(slots, generator=gen, device="cuda").to(torch.int32)
        none = torch.full((case["pad"],), -1, dtype=torch.int32, device="cuda")  # the unused end of a fixed-size list
        if op == "slot_copy":  # the n targets are no sources; several may share a source
            pick = torch.randint(0, max(1, slots - n), (n,), generator=gen, device="cuda")
            st["src"] = torch.cat([order[n:][pick] if slots > n else order[:n], none]).contiguous()
            st["dst"] = torch.cat([order[:n], none]).contiguous()
        elif op == "slot_fork":
            st["table"] = order[:n].contiguous()
            st["parents"] = torch.randint(0, n, (n,), generator=gen, device="cuda", dtype=torch.int32)
        elif op == "slot_compact":
            st["live"] = torch.zeros(slots, dtype=torch.int32, device="cuda")
            st["live"][order[:n].long()] = 1
        else:
            st["idx"] = torch.cat([order[:n], none]).contiguous()
            st["live"] = torch.ones(slots, dtype=torch.int32, device="cuda")
    return st


# ---- the plain forms -------------------------------------------------------------------------------------------


def _valid(lens, B, S):
    """(B, S): which tokens count."""
    t = torch.arange(S, device="cuda")
    return (t < lens.long()[:, None]) if lens is not None else torch.ones((B, S), dtype=torch.bool, device="cuda")


def _doubling(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 2 from h_{-1} = 0, by doubling the span that each entry covers."""
    d, S = 1, a.shape[2]
    while d < S:
        b = torch.cat([b[:, :, :d], b[:, :, d:] + a[:, :, d:] * b[:, :, :-d]], dim=2)
        a = torch.cat([a[:, :, :d], a[:, :, d:] * a[:, :, :-d]], dim=2)
        d *= 2
    return b


def _terms(x, g, valid, mix):
    """decay a and write b of every token in fp32 (a = 1, b = 0 behind the end), and x, g as they count."""
    zero = torch.zeros((), device="cuda")
    x, g = torch.where(valid, x.float(), zero), torch.where(valid, g.float(), zero)
    return torch.exp(g), (-torch.expm1(g) * x if mix else x), x, g


def _scan(x, g, h0, lens, mix):
    """every state and the last one, fp32"""
    B, N, S, D = x.shape
    valid = _valid(lens, B, S)[:, None, :, None]
    a, b, _, _ = _terms(x, g, valid, mix)
    if h0 is not None:
        b = torch.cat([b[:, :, :1] + a[:, :, :1] * h0[:, :, None], b[:, :, 1:]], dim=2)
    h = _doubling(a, b)
    return h, h[:, :, -1].clone()


def _plain_scan_fwd(s, case):
    x = s["x"]
    h, final = _scan(x, s["g"], s["h0"], s["lens"], case["mix"])
    valid = _valid(s["lens"], x.shape[0], x.shape[2])[:, None, :, None]
    return {"out": torch.where(valid, h, torch.zeros((), device="cuda")).to(x.dtype), "final_state": final}


def _plain_scan_bwd(s, case):
    x, g, h0 = s["x"], s["g"], s["checkpoints"][:, :, 0]
    B, N, S, D = x.shape
    valid = _valid(s["lens"], B, S)[:, None, :, None]
    h, _ = _scan(x, g, h0, s["lens"], case["mix"])
    before = torch.cat([h0[:, :, None], h[:, :, :-1]], dim=2)
    a, _, xf, gf = _terms(x, g, valid, case["mix"])
    zero = torch.zeros((), device="cuda")
    d = torch.where(valid, s["dout"].float(), zero)
    d = torch.cat([d[:, :, :-1], d[:, :, -1:] + s["dfinal"][:, :, None]], dim=2)
    later = torch.cat([a[:, :, 1:], torch.ones_like(a[:, :, :1])], dim=2)  # what token t + 1 passes back to t
    lam = _doubling(later.flip(2), d.flip(2)).flip(2)
    mu = a * lam
    dx = -torch.expm1(gf) * lam if case["mix"] else lam
    dg = mu * (before - xf) if case["mix"] else mu * before
    return {"dx": torch.where(valid, dx, zero).to(x.dtype), "dg": torch.where(valid, dg, zero).to(g.dtype),
            "dinitial_state": mu[:, :, 0].clone()}


def _plain_scan_step(s, case):
    x, g, pool = s["x"], s["g"], s["pool"]
    B, N, S, D = x.shape
    idx = s["idx"].long().view(B, S)
    lens = s["lens"].long() if s["lens"] is not None else torch.full((B,), S, device="cuda")
    at = s["accepted"].long() - 1 if case["per_token"] else torch.zeros(B, dtype=torch.long, device="cuda")
    h0 = pool[idx.gather(1, at[:, None])[:, 0]]
    h, _ = _scan(x, g, h0, lens, case["mix"])
    valid = _valid(lens, B, S)
    t = torch.arange(S, device="cuda")
    # a token's state is kept unless a later token of its sequence writes the same slot
    again = (idx[:, :, None] == idx[:, None, :]) & valid[:, None, :] & (t[None, None, :] > t[None, :, None])
    keep = valid & ~again.any(2)
    pool[idx[keep]] = h.transpose(1, 2)[keep]
    out = torch.where(valid[:, None, :, None], h, torch.zeros((), device="cuda")).to(x.dtype)
    return {"out": out, "state_pool": pool}


def _whole(pools):
    """the pools' contents as whole numbers: a copy is right to the last bit or wrong"""
    return [p.view(torch.int32 if p.dtype == torch.float32 else torch.int16) for p in pools]


def _plain_slot_copy(s, case):
    src, dst = s["src"], s["dst"]
    use = (src >= 0) & (dst >= 0)
    src, dst = src[use].long(), dst[use].long()
    for p in s["pools"]:
        p[dst] = p[src]
    return {"pools": _whole(s["pools"])}


def _plain_slot_fork(s, case):
    """The lowest child of a row keeps its slot; the others, in order, take the slots of the rows without a child."""
    table, par = s["table"], s["parents"].long()
    n = table.numel()
    row = torch.arange(n, device="cuda")
    first = torch.full((n,), n, device="cuda").scatter_reduce(0, par, row, "amin")
    extra, dead = row[first[par] != row], row[first == n]
    new = table[par].clone()
    new[extra] = table[dead]
    src, dst = table[par[extra]].long(), table[dead].long()
    for p in s["pools"]:
        p[dst] = p[src]
    return {"pools": _whole(s["pools"]), "slot_table": new}


def _plain_slot_compact(s, case):
    """The live slots behind the first n_live places move, in order, into the free slots before it."""
    live = s["live"] != 0
    slot = torch.arange(live.numel(), device="cuda")
    n_live = live.sum()
    src, dst = slot[live & (slot >= n_live)], slot[~live & (slot < n_live)]
    new = torch.where(live, slot, torch.full_like(slot, -1))
    new[src] = dst
    for p in s["pools"]:
        p[dst] = p[src]
    return {"pools": _whole(s["pools"]), "new_slot": new.to(torch.int32), "n_live": n_live.to(torch.int32).reshape(1)}


def _plain_slot_free(s, case):
    idx = s["idx"][s["idx"] >= 0].long()
    for p in s["pools"]:
        p[idx] = 0
    s["live"][idx] = 0
    return {"pools": _whole(s["pools"]), "live": s["live"]}


def _channels_last(q, k, v):
    """(B, N, S, D) of q, k and v -> (B, S, C)"""
    return torch.cat([t.transpose(1, 2).reshape(t.shape[0], t.shape[2], -1) for t in (q, k, v)], dim=2)


def _plain_conv1d_bwd(s, case):
    x, K = s["x"], case["K"]
    B, S, C = x.shape
    w = s["weight"].float()
    valid = _valid(s["lens"], B, S)[:, :, None]
    zero = torch.zeros((), device="cuda")
    past = s["conv_state"].float().transpose(1, 2) if s["conv_state"] is not None else torch.zeros((B, K, C), device="cuda")
    win = torch.cat([past, torch.where(valid, x.float(), zero)], dim=1).unfold(1, K, 1)[:, 1:]  # (B, S, C, K)
    pre = (win * w).sum(3) + (s["bias"].float() if s["bias"] is not None else 0.0)
    sig = torch.sigmoid(pre)
    dy = _channels_last(s["dq"], s["dk"], s["dv"]).float()
    dpre = torch.where(valid, dy * sig * (1.0 + pre * (1.0 - sig)), zero)
    ends = torch.zeros((B, K, C), device="cuda")
    dhist = torch.cat([ends, dpre, ends[:, :K - 1]], dim=1).unfold(1, K, 1)  # entry i: tokens i - K .. i - 1
    dhist = (dhist * w.flip(1)).sum(3)  # gradient of the history: K places of the state, then x
    if s["dstate_out"] is not None:  # the new state is the history from place L on
        lens = s["lens"].long() if s["lens"] is not None else torch.full((B,), S, device="cuda")
        at = (lens[:, None] + torch.arange(K, device="cuda"))[:, :, None].expand(B, K, C)
        dhist = dhist.scatter_add(1, at, s["dstate_out"].float().transpose(1, 2))
    return {"dx": torch.where(valid, dhist[:, K:], zero).to(x.dtype), "dweight": (win * dpre[..., None]).sum((0, 1)),
            "dbias": dpre.sum((0, 1)), "dconv_state": dhist[:, :K].transpose(1, 2).to(x.dtype).contiguous()}


# ---- the library's calls -----------------------------------------------------------------------------------------


def _call(s, case):
    import gated_deltanet_gdr_b200 as gdr

    op = case["op"]
    if op == "scan_fwd":
        out, final, _ = gdr.scan_fwd(s["x"], s["g"], s["h0"], s["lens"], mix=case["mix"])
        return {"out": out, "final_state": final}
    if op == "scan_bwd":
        dx, dg, dinitial = gdr.scan_bwd(s["x"], s["g"], s["checkpoints"], s["dout"], s["dfinal"], s["lens"], mix=case["mix"])
        return {"dx": dx, "dg": dg, "dinitial_state": dinitial}
    if op == "scan_step":
        out, pool = gdr.scan_step(s["x"], s["g"], s["pool"], s["idx"], s["lens"], s["accepted"], mix=case["mix"],
                                  per_token=case["per_token"])
        return {"out": out, "state_pool": pool}
    if op == "slot_copy":
        return {"pools": _whole(gdr.slot_copy(s["pools"], s["src"], s["dst"]))}
    if op == "slot_fork":
        table = gdr.slot_fork(s["pools"], s["table"], s["parents"])
        return {"pools": _whole(s["pools"]), "slot_table": table}
    if op == "slot_compact":
        new_slot, n_live = gdr.slot_compact(s["pools"], s["live"])
        return {"pools": _whole(s["pools"]), "new_slot": new_slot, "n_live": n_live}
    if op == "slot_free":
        return {"pools": _whole(gdr.slot_free(s["pools"], s["idx"], s["live"])), "live": s["live"]}
    dx, dweight, dbias, dstate = gdr.conv1d_bwd(s["x"], s["weight"], s["dq"], s["dk"], s["dv"], s["bias"], s["conv_state"],
                                                s["lens"], s["dstate_out"])
    return {"dx": dx, "dweight": dweight, "dbias": dbias, "dconv_state": dstate}


def run(state):
    case = state["case"]
    if own:
        return _call(state, case)
    plain = {"scan_fwd": _plain_scan_fwd, "scan_bwd": _plain_scan_bwd, "scan_step": _plain_scan_step,
             "slot_copy": _plain_slot_copy, "slot_fork": _plain_slot_fork, "slot_compact": _plain_slot_compact,
             "slot_free": _plain_slot_free, "conv1d_bwd": _plain_conv1d_bwd}
    return plain[case["op"]](state, case)


# ---- what a pass cannot do without ---------------------------------------------------------------------------------


def work(case):
    op = case["op"]
    if op in ("scan_fwd", "scan_bwd"):
        B, N, S, D = case["B"], case["N"], case["S"], case["D"]
        sx, sg = _bytes(case["dtype"]), _bytes(case["gate"])
        read, full = N * D * sum(_lengths(B, S, case["ragged"])), B * N * S * D  # padding is written, never read
        states = 4 * B * N * D
        if op == "scan_fwd":
            return {"bytes": read * (sx + sg) + full * sx + states * (2 if case["h0"] else 1), "flops": 3 * read}
        return {"bytes": read * (2 * sx + sg) + full * (sx + sg) + states * (2 + -(-S // CHUNK)), "flops": 10 * read}
    if op == "scan_step":
        B, N, S, D = case["B"], case["N"], case["S"], case["D"]
        tokens = B * (S + 1) / 2 if case["per_token"] else B * S
        kept = tokens if case["per_token"] else B
        return {"bytes": N * D * (tokens * (_bytes(case["dtype"]) + _bytes(case["gate"])) + B * S * _bytes(case["dtype"]) + 4 * (B + kept)),
                "flops": 3 * tokens * N * D}
    if op == "conv1d_bwd":
        C = 2 * case["Nk"] * case["Dk"] + case["Nv"] * case["Dv"]
        e, K, B, S = _bytes(case["dtype"]), case["K"], case["B"], case["S"]
        read = C * sum(_lengths(B, S, case["ragged"]))
        states = e * B * C * K * (3 if case["state"] else 1)
        return {"bytes": e * (2 * read + B * S * C) + states + C * K * (e + 4) + C * (e + 4), "flops": read * (6 * K + 12)}
    slot = _bytes(case["state"]) * (case["Nv"] * case["Dk"] * case["Dv"] + case["C"] * case["K"])
    n, slots = case["n"], case["slots"]
    if op == "slot_copy":  # every target is written, every different source read
        others = max(1, slots - n)
        moved = n + others * (1 - (1 - 1 / others) ** n)
    elif op == "slot_fork":  # the rows without a child are written, the rows with two or more read
        moved = n * (1 - 1 / n) ** n + n * (1 - (1 - 1 / n) ** n - (1 - 1 / n) ** (n - 1)) if n > 1 else 0
    elif op == "slot_compact":
        moved = 2 * n * (1 - n / slots)
    else:
        moved = n
    return {"bytes": max(1, int(moved * slot)) + 8 * n + 4 * slots, "flops": 0}


# ---- the definitions in fp64 -----------------------------------------------------------------------------------------


def _tokens(s, case, h0, lens):
    """The recurrence one token after the other in fp64: the states before and after every token."""
    x, g = s["x"], s["g"]
    h = h0.double().clone()
    before, after = [], []
    for t in range(x.shape[2]):
        on = (t < lens)[:, None, None]
        a = torch.exp(g[:, :, t].double())
        b = (1.0 - a) * x[:, :, t].double() if case["mix"] else x[:, :, t].double()
        before.append(h)
        h = torch.where(on, a * h + b, h)
        after.append(h)
    return before, after


def _exact_scan(case, s):
    B, N, S, D = s["x"].shape
    lens = s["lens"].long() if s["lens"] is not None else torch.full((B,), S, device="cuda")
    if case["op"] == "scan_step":
        idx = s["idx"].long().view(B, S)
        at = (s["accepted"].long() - 1) if case["per_token"] else torch.zeros(B, dtype=torch.long, device="cuda")
        pool = s["pool"].double()
        before, after = _tokens(s, case, pool[idx[torch.arange(B, device="cuda"), at]], lens)
        for t in range(S):
            on = t < lens
            pool[idx[on, t]] = after[t][on]
        on = _valid(lens, B, S)[:, None, :, None]
        return {"out": torch.where(on, torch.stack(after, 2), 0.0), "state_pool": pool}
    h0 = s["h0"] if s["h0"] is not None else torch.zeros((B, N, D), device="cuda")
    before, after = _tokens(s, case, h0, lens)
    if case["op"] == "scan_fwd":
        out = torch.stack([torch.where((t < lens)[:, None, None], after[t], 0.0) for t in range(S)], 2)
        return {"out": out, "final_state": after[-1]}
    mu = s["dfinal"].double()
    dx = torch.zeros((B, N, S, D), dtype=torch.float64, device="cuda")
    dg = torch.zeros_like(dx)
    for t in reversed(range(S)):
        on = (t < lens)[:, None, None]
        a = torch.exp(s["g"][:, :, t].double())
        lam = s["dout"][:, :, t].double() + mu
        x = s["x"][:, :, t].double()
        dx[:, :, t] = torch.where(on, (1.0 - a) * lam if case["mix"] else lam, 0.0)
        dg[:, :, t] = torch.where(on, a * lam * (before[t] - x if case["mix"] else before[t]), 0.0)
        mu = torch.where(on, a * lam, mu)
    return {"dx": dx, "dg": dg, "dinitial_state": mu}


def _exact_conv1d_bwd(case, s):
    x, w, K = s["x"], s["weight"].double(), case["K"]
    B, S, C = x.shape
    lens = _lengths(B, S, case["ragged"])
    dw, db = torch.zeros((C, K), dtype=torch.float64, device="cuda"), torch.zeros(C, dtype=torch.float64, device="cuda")
    dx = torch.zeros((B, S, C), dtype=torch.float64, device="cuda")
    dstate = torch.zeros((B, C, K), dtype=torch.float64, device="cuda")
    for b in range(B):
        L = lens[b]
        hist = torch.zeros((K + L, C), dtype=torch.float64, device="cuda")
        if s["conv_state"] is not None:
            hist[:K] = s["conv_state"][b].double().T
        hist[K:] = x[b, :L].double()
        pre = torch.zeros((L, C), dtype=torch.float64, device="cuda")
        for j in range(K):
            pre += w[:, j] * hist[1 + j:1 + j + L]
        if s["bias"] is not None:
            pre += s["bias"].double()
        sig = 1.0 / (1.0 + torch.exp(-pre))
        dy = torch.cat([t[b, :, :L].double().transpose(0, 1).flatten(1) for t in (s["dq"], s["dk"], s["dv"])], dim=1)
        dpre = dy * (sig + pre * sig * (1.0 - sig))
        dhist = torch.zeros_like(hist)
        for j in range(K):
            dhist[1 + j:1 + j + L] += w[:, j] * dpre
            dw[:, j] += (dpre * hist[1 + j:1 + j + L]).sum(0)
        db += dpre.sum(0)
        if s["dstate_out"] is not None:
            dhist[L:] += s["dstate_out"][b].double().T
        dx[b, :L] = dhist[K:]
        dstate[b] = dhist[:K].T
    return {"dx": dx, "dweight": dw, "dbias": db, "dconv_state": dstate}


def exact(case, seed):
    if case["op"].startswith("slot_"):
        return None  # copies: their outputs are whole numbers
    s = prepare(case, seed)
    if case["op"] == "conv1d_bwd":
        return _exact_conv1d_bwd(case, s)
    return _exact_scan(case, s)
