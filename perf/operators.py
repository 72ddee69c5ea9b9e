"""Workloads of the positional and local-attention operators: rotary positions,
sliding-window attention with sinks (forward, training, single tokens), and the
paged cache (append, attention of new tokens over the pages).

With `own` false, run() computes each operator in plain torch arithmetic (32
bits; 64 for the angles), with `own` true through this package's public calls.
exact() gives the same results from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # rotary positions of a long prompt: query and key heads of a 65536-token prefill, whole head rotated
        dict(name="rope_prefill_64k", op="rope", dtype="bf16", B=1, T=65536, H=32, Hkv=8, d=128, rot=128,
             interleaved=False, scaling="none", theta=500000.0, factor=1.0, orig=0, pos0=0, inverse=False),
        # gradient of the rotation far out in a long context, odd length, part of the head, fp32
        dict(name="rope_grad_far_f32", op="rope", dtype="f32", B=2, T=4099, H=16, Hkv=2, d=64, rot=32,
             interleaved=True, scaling="yarn", theta=10000.0, factor=32.0, orig=8192, pos0=16773000, inverse=True),
        # local attention of a long prompt: 65536 tokens, window 4096, four sinks (the largest case)
        dict(name="window_prefill_64k", op="window", dtype="bf16", B=1, Tq=65536, Tkv=65536, cap=65536, H=32, Hkv=8,
             d=128, window=4096, sinks=4, pos0=0),
        # a batch of short prompts: odd length and window, groups of three query heads, head dim 64
        dict(name="window_prefill_odd", op="window", dtype="bf16", B=3, Tq=2045, Tkv=2045, cap=2045, H=12, Hkv=4, d=64,
             window=500, sinks=7, pos0=0),
        # single tokens over a contiguous 64k cache: only the window and the sinks are read
        dict(name="window_decode", op="window", dtype="bf16", B=8, Tq=1, Tkv=65537, cap=65600, H=32, Hkv=8, d=128,
             window=4096, sinks=4, pos0=65536),
        # a training step of a local layer: forward and gradients at 16384 tokens
        dict(name="window_train_16k", op="train", dtype="bf16", B=1, T=16384, H=32, Hkv=8, d=128, window=2048, sinks=4),
        # the same in fp32 at a small odd size (gradient checks, small models)
        dict(name="window_train_f32", op="train", dtype="f32", B=2, T=777, H=4, Hkv=2, d=64, window=129, sinks=2),
        # a serving step's cache update: one new token for each of 64 sequences, q and k rotated, k and v into pages
        dict(name="append_step", op="append", dtype="bf16", B=64, most_new=1, most_kv=1024, H=32, Hkv=8, d=128, page=64,
             rot=64, interleaved=False, scaling="bands", theta=500000.0, factor=8.0, orig=8192, pad=0, ragged=1),
        # chunked prefill's cache update: up to 2048 new tokens for each of 8 sequences, small pages
        dict(name="append_chunk", op="append", dtype="bf16", B=8, most_new=2048, most_kv=8192, H=32, Hkv=8, d=128, page=16,
             rot=128, interleaved=True, scaling="linear", theta=10000.0, factor=4.0, orig=0, pad=0, ragged=2),
        # chunked prefill over the pages mixed with single tokens, up to 32768 cached, no window
        dict(name="paged_chunk", op="paged", dtype="bf16", B=6, most_new=512, most_kv=32768, H=32, Hkv=8, d=128, page=64,
             window=0, sinks=0, pad=0, ragged=3),
        # one serving step of 64 sequences, single tokens, ragged lengths up to 16384, small pages
        dict(name="paged_decode", op="paged", dtype="bf16", B=64, most_new=1, most_kv=16384, H=32, Hkv=8, d=128, page=16,
             window=0, sinks=0, pad=0, ragged=4),
        # the smallest call: one token of one sequence, window 128 and four sinks over a few hundred tokens
        dict(name="paged_one", op="paged", dtype="bf16", B=1, most_new=1, most_kv=400, H=8, Hkv=2, d=64, page=32,
             window=128, sinks=4, pad=0, ragged=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    g = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    hkv = rng.choice([1, 2, 3, 4, 8])
    return g * hkv, hkv


def _rope_fields(rng, d):
    s = rng.choice(["none", "linear", "ntk", "yarn", "bands"])
    return dict(rot=rng.choice([d, d // 2, d // 4, d - 16]), interleaved=rng.random() < 0.5, scaling=s,
                theta=rng.choice([10000.0, 500000.0, 1000000.0]),
                factor=1.0 if s == "none" else rng.choice([2.0, 4.0, 8.0, 40.0]),
                orig=rng.choice([4096, 8192]) if s in ("yarn", "bands") else 0)


def draw(rng):
    while True:     # sizes whose product would pass the largest listed case are drawn again
        c = _draw(rng)
        if work(c)["flops"] <= (2e12 if c["dtype"] == "bf16" else 2e11) and work(c)["bytes"] <= 2e9:
            return c


def _draw(rng):
    op = rng.choice(["rope", "window", "window", "train", "append", "paged", "paged"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    H, Hkv = _heads(rng)
    d = rng.choice([64, 128])
    c = dict(op=op, dtype=dtype, H=H, Hkv=Hkv, d=d)
    if op == "rope":
        T = _log(rng, 1, 16384)
        c.update(B=rng.choice([1, 2, 5]), T=T, pos0=rng.choice([0, _log(rng, 1, 16000000)]), inverse=rng.random() < 0.5)
        c.update(_rope_fields(rng, d))
    elif op == "window":
        c.update(window=rng.choice([0, _log(rng, 1, 4096)]), sinks=rng.choice([0, 1, 4, rng.randint(2, 300)]))
        if rng.random() < 0.5:      # prompts
            T = _log(rng, 1, 8192 if dtype == "bf16" else 1024)
            c.update(B=rng.choice([1, 2, 3]), Tq=T, Tkv=T, cap=T, pos0=0)
        else:                       # a few tokens over a cache, or a chunk of them
            Tq = rng.choice([1, 1, 1, 2, 5, _log(rng, 1, 512)])
            past = _log(rng, 1, 65536 if dtype == "bf16" else 8192)
            c.update(B=rng.choice([1, 2, 4]), Tq=Tq, Tkv=past + Tq, cap=past + Tq + rng.randint(0, 70), pos0=past)
    elif op == "train":
        c.update(B=rng.choice([1, 2]), T=_log(rng, 1, 4096 if dtype == "bf16" else 700),
                 window=rng.choice([0, _log(rng, 1, 2048)]), sinks=rng.choice([0, 4, rng.randint(1, 200)]))
    else:
        c.update(B=rng.choice([1, 3, 8, 33]), most_new=rng.choice([1, 1, _log(rng, 2, 300)]),
                 page=rng.choice([16, 32, 64, 128]), pad=rng.choice([0, 0, 3]), ragged=rng.randrange(1 << 30))
        c["most_kv"] = c["most_new"] + _log(rng, 1, 4096 if dtype == "bf16" else 1500)
        if op == "append":
            c.update(_rope_fields(rng, d))
        else:
            c.update(window=rng.choice([0, _log(rng, 1, 2000)]), sinks=rng.choice([0, 4, rng.randint(1, 150)]))
    return c


def _lens(case):
    """New tokens and cached tokens (new ones included) of each sequence of a ragged batch."""
    r = random.Random(case["ragged"])
    new, kv = [], []
    for _ in range(case["B"]):
        # single tokens stand among the chunks, as in a server that mixes prompts and generation
        n = 1 if case["most_new"] == 1 or r.random() < 0.25 else r.randint(1, case["most_new"])
        new.append(n)
        kv.append(r.randint(max(n, case["most_kv"] // 4), case["most_kv"]))
    return new, kv


def _pairs(n, pos0, Tkv, window, sinks):
    """Visible (query, key) pairs of n queries at pos0, pos0 + 1, ... over Tkv keys."""
    t = 0
    for p in range(pos0, pos0 + n):
        hi = min(p + 1, Tkv)
        lo = max(0, p - window + 1) if window else 0
        t += max(0, hi - lo) + min(sinks, lo, hi)
    return t


def _span(n, pos0, Tkv, window, sinks):
    """Keys that at least one of these queries sees."""
    hi = min(pos0 + n, Tkv)
    lo = max(0, pos0 - window + 1) if window else 0
    return max(0, hi - lo) + min(sinks, lo, hi)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    if case["op"] == "rope":
        n = case["B"] * case["T"] * (H + Hkv)
        return {"bytes": 2 * n * d * e, "flops": 3 * n * case["rot"]}
    if case["op"] == "window":
        a = (case["Tq"], case["pos0"], case["Tkv"], case["window"], case["sinks"])
        kv = _span(*a) * Hkv * d * 2 * e
        return {"bytes": case["B"] * (kv + 2 * case["Tq"] * H * d * e), "flops": case["B"] * 4 * d * H * _pairs(*a)}
    if case["op"] == "train":
        T = case["T"]
        pairs = case["B"] * H * _pairs(T, 0, T, case["window"], case["sinks"])
        # Q, dO read, O, dQ written; K, V read, dK, dV written
        return {"bytes": case["B"] * T * (4 * H + 4 * Hkv) * d * e, "flops": 14 * d * pairs}
    new, kv = _lens(case)
    if case["op"] == "append":
        return {"bytes": sum(new) * (2 * H + 4 * Hkv) * d * e, "flops": 3 * sum(new) * (H + Hkv) * case["rot"]}
    b = f = 0
    for n, m in zip(new, kv):
        a = (n, m - n, m, case["window"], case["sinks"])
        b += _span(*a) * Hkv * d * 2 * e + 2 * n * H * d * e
        f += 4 * d * H * _pairs(*a)
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]
    H, Hkv, d = case["H"], case["Hkv"], case["d"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    st = {"case": case}
    if own:
        import landmark_guided_chunk_b200 as hsa
        st["hsa"] = hsa
    if case["op"] == "rope":
        st["Q"], st["K"] = normal(case["B"], case["T"], H, d), normal(case["B"], case["T"], Hkv, d)
        if own:
            st["rope"] = _handle(st["hsa"], case)
    elif case["op"] == "window":
        st["Q"] = normal(case["B"], case["Tq"], H, d)
        st["K"], st["V"] = normal(case["B"], case["cap"], Hkv, d), normal(case["B"], case["cap"], Hkv, d)
        if own:
            st["ws"] = st["hsa"].window_workspace(st["Q"], st["K"], case["window"], case["sinks"],
                                                  q_pos0=case["pos0"], kv_len=case["Tkv"])
    elif case["op"] == "train":
        st["Q"], st["dO"] = normal(case["B"], case["T"], H, d), normal(case["B"], case["T"], H, d)
        st["K"], st["V"] = normal(case["B"], case["T"], Hkv, d), normal(case["B"], case["T"], Hkv, d)
        if own:
            st["ws"] = st["hsa"].window_workspace(st["Q"], st["K"], case["window"], case["sinks"], backward=True)
    else:
        new, kv = st["new"], st["kv"] = _lens(case)
        page, B = case["page"], case["B"]
        need = [-(-m // page) for m in kv]
        order = torch.randperm(sum(need) + 2, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros(B, max(need), dtype=torch.int32)
        st["K"], st["V"] = normal(sum(need) + 2, page, Hkv, d), normal(sum(need) + 2, page, Hkv, d)
        order, at = order.cpu(), 0
        for b in range(B):
            table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
        st["table"] = table.cuda()
        st["q_start"] = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32).cuda()
        st["kv_len"] = torch.tensor(kv, dtype=torch.int32).cuda()
        rows = sum(new) + case["pad"]
        st["Q"] = normal(rows, H, d)
        st["O"] = torch.zeros_like(st["Q"])
        if case["op"] == "append":
            st["k"], st["v"] = normal(rows, Hkv, d), normal(rows, Hkv, d)
            if own:
                st["rope"] = _handle(st["hsa"], case)
        if own:
            st["ws"] = st["hsa"].paged_workspace(st["Q"], st["K"], st["table"], max_q=max(new), max_kv=max(kv),
                                                 window=case.get("window", 0), sinks=case.get("sinks", 0))
    return st


def _handle(hsa, c):
    return hsa.make_rope(c["rot"], theta=c["theta"], interleaved=c["interleaved"], scaling=c["scaling"],
                         factor=c["factor"], orig_len=c["orig"])


def run(st):
    return (_own if own else _plain)[st["case"]["op"]](st, st["case"])


# ------------------------------------------------------------------------------------------------ the package's calls

def _own_rope(st, c):
    return st["hsa"].rope(st["rope"], st["Q"], st["K"], pos0=c["pos0"], inverse=c["inverse"])


def _own_window(st, c):
    return st["hsa"].window_attend(st["Q"], st["K"], st["V"], c["window"], c["sinks"], q_pos0=c["pos0"],
                                   kv_len=c["Tkv"], ws=st["ws"])


def _own_train(st, c):
    O, lse = st["hsa"].window_attend(st["Q"], st["K"], st["V"], c["window"], c["sinks"], ws=st["ws"], return_lse=True)
    return (O,) + tuple(st["hsa"].window_backward(st["Q"], st["K"], st["V"], O, lse, st["dO"], c["window"], c["sinks"],
                                                  ws=st["ws"]))


def _own_append(st, c):
    Q = st["hsa"].paged_append(st["k"], st["v"], st["K"], st["V"], st["q_start"], st["kv_len"], st["table"],
                               Q=st["Q"], rope=st["rope"], Q_out=st["O"], ws=st["ws"])
    return Q, st["K"], st["V"]


def _own_paged(st, c):
    return st["hsa"].paged_attend(st["Q"], st["K"], st["V"], st["q_start"], st["kv_len"], st["table"],
                                  max_q=max(st["new"]), max_kv=max(st["kv"]), window=c["window"], sinks=c["sinks"],
                                  O=st["O"], ws=st["ws"])


_own = {"rope": _own_rope, "window": _own_window, "train": _own_train, "append": _own_append, "paged": _own_paged}


# ------------------------------------------------------------------------------------------------ plain forms

def _freqs(c, device):
    """Angle per position of each rotated pair (64 bits), and the factor on the rotated part."""
    r, theta, s = c["rot"], c["theta"], c["factor"]
    i = torch.arange(r // 2, dtype=torch.float64, device=device)
    if c["scaling"] == "ntk":
        return (theta * s ** (r / (r - 2))) ** (-2 * i / r), 1.0
    f = theta ** (-2 * i / r)
    if c["scaling"] == "linear":
        return f / s, 1.0
    if c["scaling"] == "yarn":      # pairs that turn fewer than 1 times in the old context are slowed, above 32 kept
        def pair(turns):
            return r * math.log(c["orig"] / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), r - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / s * ramp + f * (1 - ramp), 0.1 * math.log(s) + 1.0
    if c["scaling"] == "bands":     # by wavelength: long ones slowed, short ones kept, between them joined smoothly
        turns = c["orig"] * f / (2 * math.pi)
        t = (turns - 1.0) / (4.0 - 1.0)
        return torch.where(turns < 1.0, f / s, torch.where(turns > 4.0, f, (1 - t) * f / s + t * f)), 1.0
    return f, 1.0


def _turn(x, pos, c, inverse=False):
    """Rotation of x [..., T, heads, d] at positions pos [T], 32 bits with angles in 64."""
    f, m = _freqs(c, x.device)
    a = pos.to(torch.float64)[:, None, None] * f
    cos, sin = (a.cos() * m).float(), (a.sin() * m).float()
    if inverse:
        sin = -sin
    y = x.float()
    r = c["rot"]
    if c["interleaved"]:
        x1, x2 = y[..., 0:r:2], y[..., 1:r:2]
        z = torch.stack((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1).flatten(-2)
    else:
        x1, x2 = y[..., :r // 2], y[..., r // 2:r]
        z = torch.cat((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1)
    return torch.cat((z, y[..., r:]), -1).to(x.dtype)


def _plain_rope(st, c):
    pos = c["pos0"] + torch.arange(c["T"], device="cuda")
    return _turn(st["Q"], pos, c, c["inverse"]), _turn(st["K"], pos, c, c["inverse"])


def _blocks(n, pos0, Tkv, window, sinks, size=1024):
    """Blocks of queries [t0, t1) with the slice [lo, hi) of keys that their windows reach; sinks before lo apart."""
    for t0 in range(0, n, size):
        t1 = min(n, t0 + size)
        hi = min(pos0 + t1, Tkv)
        lo = min(max(0, pos0 + t0 - window + 1) if window else 0, hi)
        yield t0, t1, lo, hi, min(sinks, lo)


def _probabilities(q, k, seen):
    """softmax over the seen keys of q k^T / sqrt(d); rows that see none are zeros. Heads lead."""
    s = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(q.shape[-1])
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    z = e.sum(-1, keepdim=True)
    return e / torch.where(z == 0, torch.ones_like(z), z)


def _seen(t0, t1, pos0, keys, window, sinks):
    p = torch.arange(pos0 + t0, pos0 + t1, device=keys.device)[:, None]
    near = (p - keys < window) if window else torch.ones_like(p == keys)
    return (keys <= p) & (near | (keys < sinks))


def _attend(Q, K, V, pos0, window, sinks):
    """One sequence: Q [n, H, d] over K, V [Tkv, Hkv, d], in 32 bits."""
    n, H, d = Q.shape
    Tkv, Hkv = K.shape[0], K.shape[1]
    out = torch.zeros(n, H, d, device=Q.device)
    if Tkv == 0:
        return out
    for t0, t1, lo, hi, ns in _blocks(n, pos0, Tkv, window, sinks):
        keys = torch.cat((torch.arange(ns, device=Q.device), torch.arange(lo, hi, device=Q.device)))
        seen = _seen(t0, t1, pos0, keys, window, sinks)
        for j in range(Hkv):
            hs = slice(j * (H // Hkv), (j + 1) * (H // Hkv))
            k = torch.cat((K[:ns, j], K[lo:hi, j])).float()
            v = torch.cat((V[:ns, j], V[lo:hi, j])).float()
            P = _probabilities(Q[t0:t1, hs].float().transpose(0, 1), k, seen)
            out[t0:t1, hs] = torch.matmul(P, v).transpose(0, 1)
    return out


def _plain_window(st, c):
    Q, K, V, n = st["Q"], st["K"], st["V"], c["Tkv"]
    return torch.stack([_attend(Q[b], K[b, :n], V[b, :n], c["pos0"], c["window"], c["sinks"])
                        for b in range(c["B"])]).to(Q.dtype)


def _plain_train(st, c):
    Q, K, V, dO = st["Q"], st["K"], st["V"], st["dO"]
    T, H, Hkv, d = c["T"], c["H"], c["Hkv"], c["d"]
    O = torch.zeros(Q.shape, device="cuda")
    dQ, dK, dV = torch.zeros(Q.shape, device="cuda"), torch.zeros(K.shape, device="cuda"), torch.zeros(K.shape, device="cuda")
    for b in range(c["B"]):
        for t0, t1, lo, hi, ns in _blocks(T, 0, T, c["window"], c["sinks"]):
            keys = torch.cat((torch.arange(ns, device="cuda"), torch.arange(lo, hi, device="cuda")))
            seen = _seen(t0, t1, 0, keys, c["window"], c["sinks"])
            for j in range(Hkv):
                hs = slice(j * (H // Hkv), (j + 1) * (H // Hkv))
                k = torch.cat((K[b, :ns, j], K[b, lo:hi, j])).float()
                v = torch.cat((V[b, :ns, j], V[b, lo:hi, j])).float()
                q, do = Q[b, t0:t1, hs].float().transpose(0, 1), dO[b, t0:t1, hs].float().transpose(0, 1)
                P = _probabilities(q, k, seen)
                o = torch.matmul(P, v)
                dS = P * (torch.matmul(do, v.T) - (do * o).sum(-1, keepdim=True)) / math.sqrt(d)
                O[b, t0:t1, hs] = o.transpose(0, 1)
                dQ[b, t0:t1, hs] = torch.matmul(dS, k).transpose(0, 1)
                gk, gv = torch.matmul(dS.transpose(1, 2), q).sum(0), torch.matmul(P.transpose(1, 2), do).sum(0)
                dK[b, :ns, j] += gk[:ns]
                dK[b, lo:hi, j] += gk[ns:]
                dV[b, :ns, j] += gv[:ns]
                dV[b, lo:hi, j] += gv[ns:]
    return O.to(Q.dtype), dQ.to(Q.dtype), dK.to(Q.dtype), dV.to(Q.dtype)


def _plain_append(st, c):
    K, V, at = st["K"], st["V"], 0
    for b, (n, m) in enumerate(zip(st["new"], st["kv"])):
        pos = torch.arange(m - n, m, device="cuda")
        rows = slice(at, at + n)
        st["O"][rows] = _turn(st["Q"][rows], pos, c)
        where = st["table"][b][pos // c["page"]].long() * c["page"] + pos % c["page"]
        K.view(-1, c["Hkv"], c["d"])[where] = _turn(st["k"][rows], pos, c)
        V.view(-1, c["Hkv"], c["d"])[where] = st["v"][rows]
        at += n
    return st["O"], K, V


def _plain_paged(st, c):
    at = 0
    for b, (n, m) in enumerate(zip(st["new"], st["kv"])):
        pages = st["table"][b, :-(-m // c["page"])].long()
        k = st["K"][pages].flatten(0, 1)[:m]
        v = st["V"][pages].flatten(0, 1)[:m]
        st["O"][at:at + n] = _attend(st["Q"][at:at + n], k, v, m - n, c["window"], c["sinks"]).to(st["O"].dtype)
        at += n
    return st["O"]


_plain = {"rope": _plain_rope, "window": _plain_window, "train": _plain_train, "append": _plain_append,
          "paged": _plain_paged}


# ------------------------------------------------------------------------------------------------ 64 bits

def _exact_turn(x, pos, c, inverse):
    """The rotation as a product of complex numbers."""
    r, h = c["rot"], c["rot"] // 2
    th, s = c["theta"], c["factor"]
    w, m = [], 1.0
    for i in range(h):
        f = th ** (-2.0 * i / r)
        if c["scaling"] == "linear":
            f /= s
        elif c["scaling"] == "ntk":
            f = (th * s ** (r / (r - 2.0))) ** (-2.0 * i / r)
        elif c["scaling"] == "yarn":
            at = [r * math.log(c["orig"] / (2 * math.pi * n)) / (2 * math.log(th)) for n in (32.0, 1.0)]
            a, b = max(0, math.floor(at[0])), min(r - 1, math.ceil(at[1]))
            u = min(1.0, max(0.0, (i - a) / max(b - a, 0.001)))
            f = u * f / s + (1 - u) * f
            m = 1.0 + 0.1 * math.log(s)
        elif c["scaling"] == "bands":
            n = c["orig"] / (2 * math.pi / f)
            u = min(1.0, max(0.0, (n - 1.0) / 3.0))
            f = u * f + (1 - u) * f / s
        w.append(f)
    a = pos.double()[:, None] * torch.tensor(w, dtype=torch.float64, device=x.device)[None]
    z = torch.polar(torch.full_like(a, m), -a if inverse else a)[:, None]
    y = x.double().clone()
    one, two = (slice(0, r, 2), slice(1, r, 2)) if c["interleaved"] else (slice(0, h), slice(h, r))
    t = torch.complex(y[..., one], y[..., two]) * z
    y[..., one], y[..., two] = t.real, t.imag
    return y


def _exact_rows(q, K, V, t, p, Tkv, window, sinks):
    """Queries q [n, G, d] at positions p [n] of one kv head: attention over the keys that any of them sees."""
    first, last = int(p[0]), int(p[-1])
    u = torch.arange(0, min(last + 1, Tkv), device=q.device)
    if window:
        u = u[(u > first - window) | (u < sinks)]
    if u.numel() == 0:
        return q.new_zeros(q.shape) * V.sum()
    k, v = K[u], V[u]
    s = torch.einsum("ngd,kd->gnk", q, k) * q.shape[-1] ** -0.5
    hidden = u[None] > p[:, None]
    if window:
        hidden |= (p[:, None] - u[None] >= window) & (u[None] >= sinks)
    s = torch.where(hidden[None], torch.full_like(s, -1e300), s)
    e = torch.softmax(s, -1) * (~hidden)[None]
    return torch.einsum("gnk,kd->ngd", e, v)


def _exact_attend(Q, K, V, pos0, window, sinks, step=512):
    n, H, d = Q.shape
    Hkv = K.shape[1]
    G = H // Hkv
    out = torch.zeros(n, H, d, dtype=torch.float64, device=Q.device)
    for j in range(Hkv):
        kj, vj = K[:, j].double(), V[:, j].double()
        for t in range(0, n, step):
            q = Q[t:t + step, j * G:(j + 1) * G].double()
            p = pos0 + torch.arange(t, t + q.shape[0], device=Q.device)
            out[t:t + step, j * G:(j + 1) * G] = _exact_rows(q, kj, vj, t, p, K.shape[0], window, sinks)
    return out


def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["op"] == "rope":
        pos = c["pos0"] + torch.arange(c["T"], device="cuda")
        return (_exact_turn(st["Q"], pos, c, c["inverse"]), _exact_turn(st["K"], pos, c, c["inverse"]))
    if c["op"] == "window":
        return torch.stack([_exact_attend(st["Q"][b], st["K"][b, :c["Tkv"]], st["V"][b, :c["Tkv"]], c["pos0"],
                                          c["window"], c["sinks"]) for b in range(c["B"])])
    if c["op"] == "train":      # gradients by differentiating the 64-bit forward, block by block of queries
        G, H, Hkv, T = c["H"] // c["Hkv"], c["H"], c["Hkv"], c["T"]
        O, dQ = (torch.zeros(st["Q"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
        dK, dV = (torch.zeros(st["K"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
        for b in range(c["B"]):
            for j in range(Hkv):
                hs = slice(j * G, (j + 1) * G)
                k, v = st["K"][b, :, j].double().requires_grad_(), st["V"][b, :, j].double().requires_grad_()
                for t in range(0, T, 512):
                    q = st["Q"][b, t:t + 512, hs].double().requires_grad_()
                    p = torch.arange(t, t + q.shape[0], device="cuda")
                    o = _exact_rows(q, k, v, t, p, T, c["window"], c["sinks"])
                    o.backward(st["dO"][b, t:t + 512, hs].double())
                    O[b, t:t + 512, hs], dQ[b, t:t + 512, hs] = o.detach(), q.grad
                dK[b, :, j], dV[b, :, j] = k.grad, v.grad
        return O, dQ, dK, dV
    out, at = st["O"].double(), 0
    K, V = st["K"].double(), st["V"].double()
    for b, (n, m) in enumerate(zip(st["new"], st["kv"])):
        slot = torch.arange(m, device="cuda")
        page, within = st["table"][b].long()[slot // c["page"]], slot % c["page"]
        if c["op"] == "append":
            pos = slot[m - n:]
            out[at:at + n] = _exact_turn(st["Q"][at:at + n], pos, c, False)
            K[page[m - n:], within[m - n:]] = _exact_turn(st["k"][at:at + n], pos, c, False)
            V[page[m - n:], within[m - n:]] = st["v"][at:at + n].double()
        else:
            out[at:at + n] = _exact_attend(st["Q"][at:at + n], K[page, within], V[page, within], m - n, c["window"],
                                           c["sinks"])
        at += n
    return (out, K, V) if c["op"] == "append" else out
