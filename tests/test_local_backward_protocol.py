"""The barrier protocols of the tcgen05 local attention's backward (window_dq_kernel and window_dkv_kernel in
landmark_guided_chunk_b200/csrc/window_bwd.cu), on the CPU.

Each role (loader, product issuers, elementwise warps, helper) is replayed with the kernel's phase arithmetic under
random interleavings, with one role or completion at a time made slow.  Checked: every role finishes; every waiter tests
its barrier only while the awaited phase is open or the one just completed, since a wait knows a parity only; and
every product, from its issue to its completion, finds in shared memory and TMEM the tile that it is meant to
read.  A change to the kernels' barriers, counts, stages or phases has to be mirrored here.
"""
import random

import pytest

from tests.test_local_protocol import Bar

POLL = object()      # yielded by a role that looks at several barriers in turn and found nothing to do


class Cta:
    def __init__(self, rng):
        self.rng, self.pipes, self.tma, self.mem = rng, {}, [], {}

    def bars(self, name, count, n):
        return [Bar(f"{name}[{i}]", count) for i in range(n)]

    def done(self, bar, phase, who):
        """A test of a barrier by parity."""
        assert phase <= bar.phase <= phase + 1, f"{who} tests phase {phase} of {bar.name} in phase {bar.phase}"
        return bar.phase > phase

    def load(self, bar, *places):
        """A TMA load: its places hold the new tile from now on, as far as an earlier reader may rely on them."""
        for where, what in places:
            self.mem[where] = what
        self.tma.append(bar)

    def product(self, pipe, reads, writes, commits):
        """Products of one issuer complete in order, those of two in any."""
        for where, what in reads:
            assert self.mem.get(where) == what, f"{pipe} finds {self.mem.get(where)} for {what} in {where}"
        self.pipes.setdefault(pipe, []).append((reads, writes, commits))
        for where, _ in writes:
            self.mem[where] = None          # being written

    def complete(self, pipe):
        reads, writes, commits = self.pipes[pipe].pop(0)
        for where, what in reads:
            assert self.mem.get(where) == what, f"{where} changed to {self.mem.get(where)} under {pipe} reading {what}"
        for where, what in writes:
            self.mem[where] = what
        for b in commits:
            b.arrive()

    def run(self):
        roles = dict(self.roles())
        asynchronous = ["tma"] + self.issuers
        slow = self.rng.choice(list(roles) + asynchronous + [""])
        waits = {r: None for r in roles}
        idle = skipped = 0
        while roles:
            who = self.rng.choice(list(roles) + asynchronous)
            if who == slow and skipped < 40 and self.rng.random() < 0.99:
                skipped += 1
                continue
            idle += 1
            skipped = 0 if who == slow else skipped
            assert idle < 60000, f"no progress: {waits}"
            if who == "tma":
                if self.tma:
                    self.tma.pop(self.rng.randrange(len(self.tma))).arrive()
                    idle = 0
                continue
            if who in self.issuers and who not in roles or who in self.issuers and self.rng.random() < 0.5:
                if self.pipes.get(who):
                    self.complete(who)
                    idle = 0
                continue
            if waits[who] not in (None, POLL) and not self.done(*waits[who], who):
                continue
            try:
                waits[who] = next(roles[who])
                idle = idle if waits[who] is POLL else 0
            except StopIteration:
                del roles[who], waits[who]
                idle = 0
        while any(self.pipes.values()):
            self.complete(self.rng.choice([p for p, v in self.pipes.items() if v]))


class Dq(Cta):
    """items: [tile is cut, ...] of each row tile's key tiles."""
    KST, VST, QSB = 6, 4, 4
    issuers = ["S", "dP", "dQ"]

    def __init__(self, items, rng, qsb=4):
        super().__init__(rng)
        self.items, self.QSB = items, qsb
        self.q_full, self.q_empty = Bar("q_full", 1), Bar("q_empty", 2)
        self.k_full, self.k_empty, self.land = (self.bars(n, 1, self.KST) for n in ("k_full", "k_empty", "land"))
        self.v_full, self.v_empty = (self.bars(n, 1, self.VST) for n in ("v_full", "v_empty"))
        self.s_full, self.s_empty = (self.bars(n, 1, self.QSB) for n in ("s_full", "s_empty"))
        self.ds_full = self.bars("ds_full", 8, self.QSB)
        self.dp_full, self.dp_empty = self.bars("dp_full", 1, 2), self.bars("dp_empty", 8, 2)
        self.dq_full, self.dq_empty = Bar("dq_full", 1), Bar("dq_empty", 16)

    def roles(self):
        yield "loader", self.loader()
        yield "S", self.scores()
        yield "dP", self.dps()
        yield "dQ", self.dqs()
        yield "helper", self.helper()
        for w in range(16):
            yield f"warp{w}", self.warp(w)

    def loader(self):
        nk = nv = nq = 0
        for item in self.items:
            for i, cut in enumerate(item):
                ks, vs = nk % self.KST, nv % self.VST
                if nk >= self.KST:
                    yield self.k_empty[ks], nk // self.KST - 1
                self.load(self.land[ks] if cut else self.k_full[ks], (("K", ks), nk))
                nk += 1
                if i == 0:
                    if nq > 0:
                        yield self.q_empty, nq - 1
                    self.load(self.q_full, ("Q", nq), ("dO", nq))
                    nq += 1
                if nv >= self.VST:
                    yield self.v_empty[vs], nv // self.VST - 1
                self.load(self.v_full[vs], (("V", vs), nv))
                nv += 1

    def scores(self):
        f = nq = 0
        for item in self.items:
            if not item:
                continue
            yield self.q_full, nq
            for i in range(len(item)):
                ks, sb = f % self.KST, f % self.QSB
                yield self.k_full[ks], f // self.KST
                if f >= self.QSB:
                    yield self.s_empty[sb], f // self.QSB - 1
                last = i == len(item) - 1
                self.product("S", [("Q", nq), (("K", ks), f)], [(("S", sb), ("S", f))],
                             [self.s_full[sb]] + ([self.q_empty] if last else []))
                f += 1
            nq += 1

    def dps(self):
        f = nq = 0
        for item in self.items:
            if not item:
                continue
            yield self.q_full, nq
            for i in range(len(item)):
                vs, sb = f % self.VST, f & 1
                yield self.v_full[vs], f // self.VST
                if f >= 2:
                    yield self.dp_empty[sb], f // 2 - 1
                last = i == len(item) - 1
                self.product("dP", [("dO", nq), (("V", vs), f)], [(("dP", sb), f)],
                             [self.dp_full[sb], self.v_empty[vs]] + ([self.q_empty] if last else []))
                f += 1
            nq += 1

    def dqs(self):
        f = nq = 0
        for item in self.items:
            if not item:
                continue
            if nq > 0:
                yield self.dq_empty, nq - 1
            for i in range(len(item)):
                ks, sb = f % self.KST, f % self.QSB
                yield self.ds_full[sb], f // self.QSB
                last = i == len(item) - 1
                self.product("dQ", [(("K", ks), f), (("S", sb), ("dS", f, 8))], [("acc", nq)] if last else [],
                             [self.s_empty[sb], self.k_empty[ks]] + ([self.dq_full] if last else []))
                f += 1
            nq += 1

    def helper(self):
        nk, uses = 0, [0] * self.KST
        for item in self.items:
            for cut in item:
                ks = nk % self.KST
                if cut:
                    yield self.land[ks], uses[ks]
                    uses[ks] += 1
                    assert self.mem[("K", ks)] == nk
                    self.k_full[ks].arrive()
                nk += 1

    def warp(self, w):
        pr, n, ni = w >> 3, 0, 0
        for item in self.items:
            for _ in item:
                if n & 1 == pr:
                    sb = n % self.QSB
                    yield self.s_full[sb], n // self.QSB
                    at = self.mem[("S", sb)]
                    assert at == ("S", n) or at[:2] == ("dS", n), f"S holds {at} for {n}"
                    yield self.dp_full[pr], n >> 1
                    assert self.mem[("dP", pr)] == n
                    self.dp_empty[pr].arrive()
                    at = self.mem[("S", sb)]
                    self.mem[("S", sb)] = ("dS", n, 1 + (at[2] if at[0] == "dS" else 0))
                    self.ds_full[sb].arrive()
                n += 1
            if item:
                yield self.dq_full, ni
                assert self.mem["acc"] == ni
                self.dq_empty.arrive()
                ni += 1


class Dkv(Cta):
    """items: number of row tiles of each key tile's work item."""
    RST = 4
    issuers = ["SP", "VK"]

    def __init__(self, items, rng):
        super().__init__(rng)
        self.items = items
        self.kv_full, self.kv_empty = Bar("kv_full", 1), Bar("kv_empty", 1)
        self.r_full, self.r_empty, self.st_full = (self.bars(n, 1, self.RST) for n in ("r_full", "r_empty", "st_full"))
        self.st_empty = self.bars("st_empty", 8, self.RST)
        self.s_full, self.s_empty, self.dp_full, self.dp_empty = (
            self.bars(n, 1, 2) for n in ("s_full", "s_empty", "dp_full", "dp_empty"))
        self.p_full, self.ds_full = self.bars("p_full", 8, 2), self.bars("ds_full", 8, 2)
        self.acc_full, self.acc_empty = Bar("acc_full", 1), Bar("acc_empty", 16)

    def roles(self):
        yield "loader", self.loader()
        yield "SP", self.scores_and_dps()
        yield "VK", self.dvs_and_dks()
        yield "stats", self.stats()
        for w in range(16):
            yield f"warp{w}", self.warp(w)

    def loader(self):
        ni = n = 0
        for nt in self.items:
            if nt == 0:
                continue
            if ni > 0:
                yield self.kv_empty, ni - 1
            self.load(self.kv_full, ("KV", ni))
            ni += 1
            for _ in range(nt):
                st = n % self.RST
                if n >= self.RST:
                    yield self.r_empty[st], n // self.RST - 1
                self.load(self.r_full[st], (("R", st), n))
                n += 1

    def scores_and_dps(self):
        n = ni = 0
        for nt in self.items:
            if nt == 0:
                continue
            yield self.kv_full, ni
            i_s = i_p = 0
            while i_p < nt:
                moved = False
                if i_s < nt:
                    f = n + i_s
                    st, sb = f % self.RST, f & 1
                    if self.done(self.r_full[st], f // self.RST, "SP") and (
                            f < 2 or self.done(self.s_empty[sb], f // 2 - 1, "SP")):
                        self.product("SP", [("KV", ni), (("R", st), f)], [(("S", sb), ("S", f))], [self.s_full[sb]])
                        i_s, moved = i_s + 1, True
                if i_p < i_s:
                    f = n + i_p
                    st, sb = f % self.RST, f & 1
                    if f < 2 or self.done(self.dp_empty[sb], f // 2 - 1, "SP"):
                        self.product("SP", [("KV", ni), (("R", st), f)], [(("dP", sb), ("dP", f))],
                                     [self.dp_full[sb]] + ([self.kv_empty] if i_p == nt - 1 else []))
                        i_p, moved = i_p + 1, True
                if not moved:
                    yield POLL
            n, ni = n + nt, ni + 1

    def dvs_and_dks(self):
        n = ni = 0
        for nt in self.items:
            if nt == 0:
                continue
            if ni > 0:
                yield self.acc_empty, ni - 1
            iv = ik = 0
            while ik < nt:
                moved = False
                if iv < nt:
                    f = n + iv
                    st, sb = f % self.RST, f & 1
                    if self.done(self.p_full[sb], f >> 1, "VK"):
                        self.product("VK", [(("R", st), f), (("S", sb), ("P", f, 8))], [], [self.s_empty[sb]])
                        iv, moved = iv + 1, True
                if ik < iv:
                    f = n + ik
                    st, sb = f % self.RST, f & 1
                    if self.done(self.ds_full[sb], f >> 1, "VK"):
                        last = ik == nt - 1
                        self.product("VK", [(("R", st), f), (("dP", sb), ("dS", f, 8))], [("acc", ni)] if last else [],
                                     [self.dp_empty[sb], self.r_empty[st]] + ([self.acc_full] if last else []))
                        ik, moved = ik + 1, True
                if not moved:
                    yield POLL
            n, ni = n + nt, ni + 1

    def stats(self):
        n = 0
        for nt in self.items:
            for _ in range(nt):
                st = n % self.RST
                if n >= self.RST:
                    yield self.st_empty[st], n // self.RST - 1
                self.mem[("stats", st)] = n
                self.st_full[st].arrive()
                n += 1

    def _put(self, where, name, n):
        at = self.mem[where]
        self.mem[where] = (name, n, 1 + (at[2] if at[0] == name else 0))

    def warp(self, w):
        pr, n, ni = w >> 3, 0, 0
        for nt in self.items:
            for _ in range(nt):
                if n & 1 == pr:
                    st = n % self.RST
                    yield self.st_full[st], n // self.RST
                    yield self.s_full[pr], n >> 1
                    assert self.mem[("stats", st)] == n and self.mem[("S", pr)][1] == n
                    self._put(("S", pr), "P", n)
                    self.p_full[pr].arrive()
                    yield self.dp_full[pr], n >> 1
                    assert self.mem[("stats", st)] == n and self.mem[("dP", pr)][1] == n
                    self._put(("dP", pr), "dS", n)
                    self.st_empty[st].arrive()
                    self.ds_full[pr].arrive()
                n += 1
            if nt:
                yield self.acc_full, ni
                assert self.mem["acc"] == ni
                self.acc_empty.arrive()
                ni += 1


def _lengths(rng):
    return [rng.choice([0, 1, 1, 2, 3, 9, 14]) for _ in range(rng.randint(1, 7))]


def test_dq_protocol():
    for seed in range(150):
        rng = random.Random(seed)
        Dq([[rng.random() < 0.3 for _ in range(n)] for n in _lengths(rng)], rng).run()


def test_dkv_protocol():
    for seed in range(150):
        rng = random.Random(seed)
        Dkv(_lengths(rng), rng).run()


@pytest.mark.parametrize("kind", ["k_empty", "s_empty", "dp_empty"])
def test_the_model_sees_a_missing_wait(kind):
    """The model with one role's wait for a free buffer left out."""
    class Hasty(Dq):
        def loader(self):
            return (w for w in super().loader() if kind != "k_empty" or w[0] not in self.k_empty)

        def scores(self):
            return (w for w in super().scores() if kind != "s_empty" or w[0] not in self.s_empty)

        def dps(self):
            return (w for w in super().dps() if kind != "dp_empty" or w[0] not in self.dp_empty)

    with pytest.raises(AssertionError):
        for seed in range(300):
            rng = random.Random(seed)
            Hasty([[False] * n for n in _lengths(rng)], rng).run()
