"""The barrier protocol of the tcgen05 local attention (window_fwd_kernel in
landmark_guided_chunk_b200/csrc/window_tc.cu), on the CPU.

A CTA takes work items, each of 0 to 2 row tiles against a run of key tiles.  Roles: the loader (K and V tiles into a
ring, an item's Q tiles into one of two buffers), the MMA warp, four softmax warps per row tile, the helper that zeroes
dead V rows, and the output warp, which stores an item's output from its Q buffer and frees it.  This model replays each
role with the kernel's phase arithmetic under random interleavings and completion delays, with one role at a time made
slow, and checks that every role finishes and that every waiter tests its barrier only while the awaited phase is open
or the one just completed: a wait that knows only a parity misreads anything else.

Waits are bounded in time.  A wait with the plain limit may only span a ring's worth of the loader's tiles; the roles
that pass over tiles without a wait of their own (the helper, the output warp, the softmax of the second row tile) count
their limit from the loader's last tile (mbar_wait_ahead).  A change to the kernel's barriers, counts, phases or limits
has to be mirrored here.
"""
import random

import pytest

QB = 2     # buffers of the Q tiles


class Bar:
    def __init__(self, name, count):
        self.name, self.count, self.arrived, self.phase = name, count, 0, 0

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.count:
            self.arrived, self.phase = 0, self.phase + 1


class Cta:
    """items: (row tiles, [tile has dead V rows, ...]).  Each role is a generator that yields (barrier, phase) waits."""

    def __init__(self, items, nst, rng, out_buffers=QB, ahead=("helper", "output", "softmax")):
        self.items, self.nst, self.rng, self.outs, self.ahead = items, nst, rng, out_buffers, ahead
        self.step = 0                      # tiles that the loader has issued
        def grid(name, count, *dims):
            if not dims:
                return Bar(name, count)
            return [grid(f"{name}[{i}]", count, *dims[1:]) for i in range(dims[0])]
        self.q_full, self.q_empty = grid("q_full", 1, QB, 2), grid("q_empty", 1, QB, 2)
        self.kv_full, self.kv_empty, self.land = (grid(n, 1, nst) for n in ("kv_full", "kv_empty", "land"))
        self.s_full, self.o_full = grid("s_full", 1, 2), grid("o_full", 1, 2)
        self.p_full = grid("p_full", 4, 2, 2)
        self.out_full = grid("out_full", 4, out_buffers, 2)
        self.tma, self.mma = [], []        # completions on their way: any order; in order

    def work(self):
        """Items with keys, in order; the others are passed over by every role but the softmax's zeros."""
        return [(n, dead) for n, dead in self.items if n > 0 and dead]

    def loader(self):
        nkv, na = 0, 0
        fills = [[0, 0] for _ in range(QB)]
        for ntile, tiles in self.work():
            for i, dead in enumerate(tiles):
                for kv in range(2):
                    s = nkv % self.nst
                    if nkv >= self.nst:
                        yield self.kv_empty[s], nkv // self.nst - 1
                    self.tma.append([self.land[s] if kv and dead else self.kv_full[s]])
                    nkv += 1
                    self.step = nkv
                    if kv == 0 and i == 0:
                        x, na = na % QB, na + 1
                        for t in range(ntile):
                            if fills[x][t]:
                                yield self.q_empty[x][t], fills[x][t] - 1
                            fills[x][t] += 1
                            self.tma.append([self.q_full[x][t]])

    def issuer(self):
        uses, qf, pf = [0] * self.nst, [[0, 0] for _ in range(QB)], [0, 0]
        na = head = 0
        def kv(s):
            uses[s] += 1
            return self.kv_full[s], uses[s] - 1
        for ntile, tiles in self.work():
            nt, x, na = len(tiles), na % QB, na + 1
            ks = head
            yield kv(ks)
            for t in range(ntile):
                yield self.q_full[x][t], qf[x][t]
                qf[x][t] += 1
                self.mma.append([self.s_full[t]] + ([self.kv_empty[ks]] if t == ntile - 1 else []))
            for i in range(nt):
                vs = (ks + 1) % self.nst
                kn = (vs + 1) % self.nst
                for t in range(ntile):
                    if t == 0:
                        yield kv(vs)
                    for h in range(2):
                        yield self.p_full[t][h], pf[t]
                    pf[t] += 1
                    self.mma.append([self.o_full[t]] + ([self.kv_empty[vs]] if t == ntile - 1 else []))
                    if i + 1 < nt:
                        if t == 0:
                            yield kv(kn)
                        self.mma.append([self.s_full[t]] + ([self.kv_empty[kn]] if t == ntile - 1 else []))
                ks, head = kn, (vs + 1) % self.nst

    def softmax(self, t):
        n = na = 0
        for ntile, tiles in self.items:
            any_ = bool(tiles) and ntile > 0
            if t >= ntile:
                na += any_
                continue
            for i in range(len(tiles)):
                yield self.s_full[t], n
                if i and self.rng.random() < 0.3:      # a maximum that grew
                    yield self.o_full[t], n - 1
                for h in range(2):
                    self.p_full[t][h].arrive()
                n += 1
            if any_:
                yield self.o_full[t], n - 1
                self.out_full[na % self.outs][t].arrive()
                na += 1

    def helper(self):
        nkv, uses = 0, [0] * self.nst
        for _, tiles in self.work():
            for dead in tiles:
                s = (nkv + 1) % self.nst
                nkv += 2
                if dead:
                    yield self.land[s], uses[s]
                    uses[s] += 1
                    self.kv_full[s].arrive()

    def output(self):
        na, seen = 0, [[0, 0] for _ in range(self.outs)]
        for ntile, _ in self.work():
            x, o, na = na % QB, na % self.outs, na + 1
            for t in range(ntile):
                yield self.out_full[o][t], seen[o][t]
                seen[o][t] += 1
                self.q_empty[x][t].arrive()

    def run(self):
        roles = {"loader": self.loader(), "issuer": self.issuer(), "helper": self.helper(), "output": self.output()}
        for t in range(2):
            for w in range(4):
                roles[f"softmax{t}.{w}"] = self.softmax(t)
        slow = self.rng.choice(list(roles) + ["tma", "mma", ""])
        waits = {r: None for r in roles}       # None: ready to run on
        since = {r: 0 for r in roles}
        idle = 0
        while roles:
            who = self.rng.choice(list(roles) + ["tma", "mma"])
            # the slow one moves when nothing else can, or now and then
            if who == slow and idle < 40 and self.rng.random() < 0.99:
                idle += 1
                continue
            idle += 1
            assert idle < 4000, f"no progress: {waits}"
            if who in ("tma", "mma"):
                pending = self.tma if who == "tma" else self.mma
                if pending:
                    for b in pending.pop(self.rng.randrange(len(pending)) if who == "tma" else 0):
                        b.arrive()
                    idle = 0
                continue
            if waits[who] is not None:
                bar, phase = waits[who]
                assert phase <= bar.phase <= phase + 1, f"{who} tests phase {phase} of {bar.name} in phase {bar.phase}"
                if bar.phase == phase:      # the kernel looks at its limit after a failed test
                    # (the softmax's o_full waits have the plain one)
                    if not who.startswith(self.ahead) or bar in self.o_full:
                        assert self.step - since[who] <= 2 * self.nst, f"{who}: limit spans {self.step - since[who]} tiles"
                    continue
            idle = 0
            try:
                waits[who] = next(roles[who])
                since[who] = self.step
            except StopIteration:
                del roles[who], waits[who]


def _items(rng):
    short = rng.random() < 0.5
    return [(rng.choice([0, 1, 2, 2]), [rng.random() < 0.3 for _ in range(rng.choice([0, 1, 1, 2] if short else [1, 3, 9]))])
            for _ in range(rng.randint(1, 12))]


@pytest.mark.parametrize("nst", [3, 8])    # head dim 128, 64
def test_forward_protocol(nst):
    for seed in range(1500):
        rng = random.Random(seed)
        Cta(_items(rng), nst, rng).run()


def test_one_output_barrier_per_row_tile_would_not_do():
    """With a barrier per row tile alone, the softmax can finish the next item, whose output goes to the other buffer,
    before the output warp has looked for this one's."""
    with pytest.raises(AssertionError, match="output tests phase"):
        for seed in range(1500):
            rng = random.Random(seed)
            Cta(_items(rng), 3, rng, out_buffers=1).run()


@pytest.mark.parametrize("role", ["helper", "output", "softmax"])
def test_roles_that_run_ahead_need_their_own_limit(role):
    ahead = tuple({"helper", "output", "softmax"} - {role})
    with pytest.raises(AssertionError, match=f"{role}.*: limit spans"):
        for seed in range(1500):
            rng = random.Random(seed)
            Cta(_items(rng), 3, rng, ahead=ahead).run()


def _drained(issued, landed, nst, parity_of):
    """Whether a producer that has issued that many tiles into its ring, the first `landed` of which have arrived (and
    been consumed as far as a refill needs), would go on from its drain: a wait by parity passes unless the open phase
    has it."""
    phase = [len([i for i in range(landed) if i % nst == x]) for x in range(nst)]
    return all(phase[x] & 1 != parity_of(issued, x, nst) for x in range(nst) if parity_of(issued, x, nst) is not None)


def _last_use(issued, x, nst):
    """window_few_kernel on an expired wait: the phase of a stage's last use; unused stages have none."""
    return (issued - 1 - x) // nst & 1 if x < issued else None


@pytest.mark.parametrize("nst", [3, 4, 6])
def test_a_producer_that_gives_up_waits_for_its_loads(nst):
    """Loads that are still in flight when the CTA ends would land in the next one's shared memory."""
    for issued in range(4 * nst):
        for landed in range(max(0, issued - nst), issued + 1):
            assert _drained(issued, landed, nst, _last_use) == (landed == issued), (issued, landed)
    # parity 0 for every stage passes with the second use still in flight, and waits on stages without a load
    zero = lambda issued, x, nst: 0    # noqa: E731
    assert _drained(2 * nst, nst, nst, zero) and not _drained(1, 1, nst, zero)


def _tile_by_row(q_start, x, tok):
    """tile_by_row of csrc/local.cuh: (sequence, its block) of the x-th row tile over all sequences, or None."""
    first = lambda i: q_start[i] // tok + i    # noqa: E731
    lo, hi = 0, len(q_start) - 2
    while lo < hi:
        mid = (lo + hi + 1) >> 1
        lo, hi = (mid, hi) if first(mid) <= x else (lo, mid - 1)
    return (lo, x - first(lo)) if x >= first(lo) else None


def _ragged(rng):
    n = [rng.choice([0, 1, 1, 1, 2, 7, 300]) for _ in range(rng.randint(1, 40))]
    return n, [sum(n[:i]) for i in range(len(n) + 1)]


@pytest.mark.parametrize("tok", [1, 4, 5, 32])
def test_row_tiles_over_all_sequences_cover_each_block_once(tok):
    for seed in range(100):
        n, q_start = _ragged(random.Random(seed))
        got = [_tile_by_row(q_start, x, tok) for x in range(q_start[-1] // tok + len(n))]
        live = [g for g in got if g and g[1] * tok < n[g[0]]]
        assert sorted(live) == [(b, k) for b, m in enumerate(n) for k in range(-(-m // tok))]


@pytest.mark.parametrize("grid,hkv,tok", [(148, 2, 4), (148, 8, 32), (5, 3, 1)])
def test_the_walk_past_empty_blocks_meets_every_item(grid, hkv, tok):
    """Walk::next of csrc/window_tc.cu: a sequence's blocks without tokens come first and are stepped over."""
    for seed in range(60):
        n, q_start = _ragged(random.Random(seed))
        nblk = -(-q_start[-1] // (2 * tok))
        blocks = [-(-m // (2 * tok)) for m in n]
        want = [g for g in range(len(n) * nblk * hkv) if nblk - 1 - g // hkv % nblk < blocks[g // hkv // nblk]]
        got, looks = [], 0
        for g in range(grid):
            while g < len(n) * nblk * hkv:
                b, on = g // hkv // nblk, 1
                looks += 1
                if nblk - 1 - g // hkv % nblk < blocks[b]:
                    got.append(g)
                else:
                    on += ((b * nblk + nblk - blocks[b]) * hkv - g - 1) // grid
                    assert on >= 1
                g += on * grid
        assert sorted(got) == want and looks <= len(want) + len(n) * grid
