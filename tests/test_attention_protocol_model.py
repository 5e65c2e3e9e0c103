"""A CPU model of the attention kernel's barrier protocol (attention.cuh): no
deadlock, no parity aliasing, and an order of items that misses none.

The kernel's roles -- items, loads, MMA issue and softmax of two streams,
epilogue -- hand work on through mbarriers that are waited on by phase parity.
A parity wait passes once the phase of that parity has completed: on a barrier
that has run a phase too few it can pass at once, and on one that has run a
phase too many it hangs.  The model replays each role's loops with the
kernel's own parities beside an independent count of which completion each
wait is meant to see.  Copies land and MMAs complete at random times (MMAs of
one thread in order), warps advance in random order; every run must finish and
every wait must see exactly the completion it means.  Two arrangements the
kernel does not have are planted to show that the model notices them.
"""
import random

import pytest

SLOTS = 3  # item descriptors in flight


class Bar:
    def __init__(self, count):
        self.count, self.arrived, self.done = count, 0, 0

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.count:
            self.arrived, self.done = 0, self.done + 1

    def passes(self, parity):
        return (self.done & 1) != parity


def tiles_of(item, t):
    return item["n0"] if t == 0 else (item["n"] // 2 if item["solo"] else item["n"])


def walk(n):
    """Key and value tiles in ring order: (is key, tile)."""
    keys = values = 0
    while keys + values < 2 * n:
        if keys < n and (keys < 2 or keys <= values + 1):
            yield True, keys
            keys += 1
        else:
            yield False, values
            values += 1


class Model:
    """One CTA working through `items`; warps: softmax and epilogue warps of a role."""

    def __init__(self, items, ring, turns, seed, one_tail=False, skip_foreign=False, warps=2):
        self.items, self.ring, self.turns, self.warps = items, ring, turns, warps
        self.one_tail, self.skip_foreign = one_tail, skip_foreign
        self.rng = random.Random(seed)
        b = self.bars = {}
        for s in range(ring):
            b["full", s] = Bar(1)
            b["empty", s] = Bar(1 if skip_foreign else 2)
        for t in range(2):
            for name, count in (("qfull", 1), ("qempty", 1), ("sfull", 1), ("ofull", 1), ("p0", warps), ("p1", warps),
                                ("mlfull", warps), ("mlempty", warps), ("oempty", warps), ("turn", warps)):
                b[name, t] = Bar(count)
        for s in range(SLOTS):
            b["item", s] = Bar(1)
            b["free", s] = Bar(2 * warps + warps + 2 + 1)
            b["tail", s] = Bar(1)
            b["fixed", s] = Bar(warps)
        b["ask", 0] = Bar(1)
        self.landing = []        # copies in flight: barriers that will be arrived on
        self.pipe = [[], []]     # commits of each MMA thread, in order

    # -- roles: generators yielding (barrier, parity, completion meant) --------
    def item_wait(self, it):
        return ("item", it % SLOTS), (it // SLOTS) & 1, it // SLOTS

    def role_items(self):
        for it in range(len(self.items) + 1):
            yield ("free", it % SLOTS), ((it // SLOTS) & 1) ^ 1, it // SLOTS - 1
            self.bars["item", it % SLOTS].arrive()
            if it < len(self.items):
                yield ("ask", 0), it & 1, it

    def role_loads(self):
        base, nq = 0, [0, 0]
        for it, item in enumerate(self.items):
            yield self.item_wait(it)
            n = item["n"]
            for pos, (is_key, j) in enumerate(walk(n)):
                if pos == 1:
                    for t in range(2):
                        if tiles_of(item, t):
                            yield ("qempty", t), (nq[t] & 1) ^ 1, nq[t] - 1
                            nq[t] += 1
                            self.landing.append(("qfull", t))
                if pos == max(2 * n - 4, 0):
                    self.bars["ask", 0].arrive()
                g = base + pos
                yield ("empty", g % self.ring), ((g // self.ring) & 1) ^ 1, g // self.ring - 1
                self.landing.append(("full", g % self.ring))
            base += 2 * n
            if n == 0:
                self.bars["ask", 0].arrive()
            self.bars["free", it % SLOTS].arrive()

    def role_mma(self, t):
        base = nq = np = no = 0
        for it, item in enumerate(self.items):
            slot, phase = it % SLOTS, (it // SLOTS) & 1
            yield self.item_wait(it)
            n, solo, fix, cnt = item["n"], item["solo"], item["fix"], tiles_of(item, t)
            teller = t == (((n - 1) & 1) if solo else 1)
            tail = ("tail", 0 if self.one_tail else slot)
            if teller and not fix and not self.one_tail:
                self.bars[tail].arrive()
            keys, vtile, vslot, kslot, key = 0, -1, 0, 0, False
            for pos, (is_key, j) in enumerate(walk(n)):
                g = base + pos
                rslot = g % self.ring
                foreign = (j & 1) != t if solo else j >= cnt
                if foreign and self.skip_foreign:
                    continue
                yield ("full", rslot), (g // self.ring) & 1, g // self.ring
                if foreign:
                    self.bars["empty", rslot].arrive()
                    continue
                if is_key:
                    kslot, key, keys = rslot, True, keys + 1
                else:
                    vslot, vtile = rslot, j
                if (keys != 1) if vtile < 0 else (not key and keys < cnt):
                    continue
                if vtile < 0:
                    yield ("qfull", t), nq & 1, nq
                    nq += 1
                else:
                    if fix and vtile == n - 1:
                        if teller:
                            self.bars[tail].arrive()
                        yield ("fixed", slot), phase, it // SLOTS
                    first = vtile < (2 if solo else 1)
                    if first:
                        yield ("oempty", t), (no & 1) ^ 1, no - 1
                        no += 1
                    yield ("p0", t), np & 1, np
                    yield ("p1", t), np & 1, np
                    np += 1
                    self.pipe[t].append(("empty", vslot))
                    if not key:
                        self.pipe[t].append(("ofull", t))
                    vtile = -1
                if key:
                    key = False
                    self.pipe[t].append(("sfull", t))
                    self.pipe[t].append(("empty", kslot))
                    if keys == cnt:
                        self.pipe[t].append(("qempty", t))
            base += 2 * n
            self.bars["free", slot].arrive()

    def role_softmax(self, t):
        nscore = nml = nturn = 0
        for it, item in enumerate(self.items):
            yield self.item_wait(it)
            cnt = tiles_of(item, t)
            common = item["n0"] if self.turns and not item["solo"] else 0
            for i in range(cnt):
                yield ("sfull", t), nscore & 1, nscore
                nscore += 1
                if i < common:
                    yield ("turn", t), (nturn & 1) ^ (t == 0), nturn - (t == 0)
                    nturn += 1
                self.bars["p0", t].arrive()
                yield None
                self.bars["p1", t].arrive()
                if i < common:
                    self.bars["turn", 1 - t].arrive()
            if cnt:
                yield ("mlempty", t), (nml & 1) ^ 1, nml - 1
                nml += 1
                self.bars["mlfull", t].arrive()
            self.bars["free", it % SLOTS].arrive()

    def role_epilogue(self):
        nout, tails = [0, 0], 0
        for it, item in enumerate(self.items):
            slot, phase = it % SLOTS, (it // SLOTS) & 1
            yield self.item_wait(it)
            if self.one_tail:  # (a single barrier, arrived on only where there is a tail)
                if item["fix"]:
                    yield ("tail", 0), tails & 1, tails
                    tails += 1
            else:
                yield ("tail", slot), phase, it // SLOTS
            self.bars["fixed", slot].arrive()
            solo, n = item["solo"], item["n"]
            for t in range(1 if solo else 2):
                for u in ((0, 1) if solo and n > 1 else (t,)):
                    if tiles_of(item, u):
                        yield ("mlfull", u), nout[u] & 1, nout[u]
                        self.bars["mlempty", u].arrive()
                        yield ("ofull", u), nout[u] & 1, nout[u]
                        nout[u] += 1
                for u in ((0, 1) if solo and n > 1 else (t,)):
                    if tiles_of(item, u):
                        self.bars["oempty", u].arrive()
            self.bars["free", slot].arrive()

    def run(self):
        roles = [self.role_items(), self.role_loads(), self.role_mma(0), self.role_mma(1)]
        roles += [self.role_softmax(t) for t in range(2) for _ in range(self.warps)]
        roles += [self.role_epilogue() for _ in range(self.warps)]
        waits = [next(r) for r in roles]
        live = set(range(len(roles)))
        # each run favours some roles and events, so that they lag or lead by much
        weight = [self.rng.choice((0.05, 1, 1, 20)) for _ in roles]
        land, finish = self.rng.choice((0.02, 1, 10)), [self.rng.choice((0.05, 1, 10)) for _ in range(2)]
        while live:
            ready = [i for i in live if waits[i] is None or self.bars[waits[i][0]].passes(waits[i][1])]
            moves = [(weight[i], ("role", i)) for i in ready]
            if self.landing:
                moves.append((land, ("land", 0)))
            moves += [(finish[t], ("mma", t)) for t in range(2) if self.pipe[t]]
            assert moves, f"deadlock: {sorted(str(waits[i]) for i in live)}"
            _, (kind, i) = self.rng.choices(moves, [m[0] for m in moves])[0]
            if kind == "land":
                self.bars[self.landing.pop(self.rng.randrange(len(self.landing)))].arrive()
            elif kind == "mma":
                self.bars[self.pipe[i].pop(0)].arrive()
            else:
                if waits[i] is not None:
                    bar, _, meant = waits[i]
                    assert self.bars[bar].done == meant + 1, f"{bar}: completion {meant} meant, {self.bars[bar].done} seen"
                try:
                    waits[i] = next(roles[i])
                except StopIteration:
                    live.discard(i)
        assert not self.landing and not self.pipe[0] and not self.pipe[1]


def random_items(rng, count):
    out = []
    for _ in range(count):
        n = rng.choice((0, 1, 1, 2, 2, 3, 4, 5, 7, 9))
        solo = rng.random() < 0.5
        n0 = (n + 1) // 2 if solo else max(0, n - rng.choice((0, 0, 1, 2, 9)))
        out.append(dict(n=n, solo=solo, n0=n0, fix=n > 0 and rng.random() < 0.6))
    return out


@pytest.mark.parametrize("ring,turns", [(5, True), (8, False)])  # 128- and 64-wide heads
def test_no_deadlock_and_no_aliasing(ring, turns):
    rng = random.Random(ring)
    for seed in range(250):
        Model(random_items(rng, rng.choice((1, 2, 6, 14))), ring, turns, seed).run()


@pytest.mark.parametrize("planted", ["one_tail", "skip_foreign"])
def test_the_model_notices_planted_mistakes(planted):
    """One barrier for the tails of all items; streams that leave out the ring tiles they do not use."""
    rng = random.Random(7)
    with pytest.raises(AssertionError):
        for seed in range(400):
            Model(random_items(rng, 14), 5, False, seed, **{planted: True}).run()


# ------------------------------------------------------------ order of items --
class Search:
    """The kernel's search for an item number (decode_item), with the cursor that a CTA keeps."""

    def __init__(self, seqs, block, causal, tile=128):
        self.seqs, self.block, self.causal, self.tile = seqs, block, causal, tile
        self.most = -(-sum(k for _, k in seqs) // tile)
        self.reset()

    def reset(self):
        self.n = self.first = self.end = self.seq0 = self.before = 0
        self.all = -1

    def blocks(self, q):
        return -(-q // self.block)

    def count(self, s, n):
        q, k = s
        keys = (n - 1) * self.tile + 1
        if n == 0:
            return self.blocks(q)
        if k < keys:
            return 0
        if not self.causal:
            return self.blocks(q)
        return self.blocks(q) - max(self.blocks(max(keys - (k - q), 0)) - 1, 0)

    def counts(self, n):
        return sum(self.count(s, n) for s in self.seqs)

    def find(self, u):
        """(sequence, block) of item u, or None."""
        if u < self.first or u >= self.end:
            if self.all < 0:
                self.all = self.counts(0)
                self.n = -(-max(k for _, k in self.seqs) // self.tile) + 1
            if u >= self.all:
                return None
            lo, hi, more, whole = 0, self.n, self.end, self.all
            if u < self.first:
                hi, more = self.most + 1, 0
            while hi - lo > 1:
                mid = (lo + hi) // 2
                n = self.counts(mid)
                if n > u:
                    lo, whole = mid, n
                else:
                    hi, more = mid, n
            self.n, self.first, self.end, self.seq0, self.before = lo, more, whole, 0, 0
        elif u < self.first + self.before:
            self.seq0 = self.before = 0
        u -= self.first + self.before
        while self.seq0 < len(self.seqs):
            for b, s in enumerate(self.seqs[self.seq0:self.seq0 + 32], self.seq0):
                here = self.count(s, self.n) - self.count(s, self.n + 1)
                if u < here:
                    return b, self.blocks(s[0]) - self.count(s, self.n) + u
                u -= here
            self.before += sum(self.count(s, self.n) - self.count(s, self.n + 1) for s in self.seqs[self.seq0:self.seq0 + 32])
            self.seq0 += 32
        raise AssertionError("no sequence holds the item")


def enumerate_items(seqs, block, causal):
    """Every item, each searched for from the beginning."""
    out, search = [], Search(seqs, block, causal)
    while (item := search.find(len(out))) is not None:
        out.append(item)
        search.reset()
    return out


def test_items_found_from_the_one_before():
    """A CTA's numbers mostly rise, by any step; whatever they do, it finds what a fresh search finds."""
    rng = random.Random(5)
    for _ in range(200):
        seqs = [(rng.choice((0, 1, rng.randint(0, 500))), rng.choice((0, 1, rng.randint(0, 900))))
                for _ in range(rng.choice((1, 5, 31, 32, 33, 64, 100)))]
        block, causal = rng.choice((18, 32, 64, 256)), rng.random() < 0.7
        want = enumerate_items(seqs, block, causal)
        search, u = Search(seqs, block, causal), rng.randint(0, 20)
        for _ in range(60):
            assert search.find(u) == (want[u] if u < len(want) else None)
            u = max(0, u + rng.choice((0, 1, 1, 3, 19, 40, -1, -7, -len(want))))


def test_every_block_is_an_item_and_the_longest_come_first():
    rng = random.Random(3)
    for _ in range(300):
        seqs = [(rng.choice((0, 1, rng.randint(0, 900))), rng.choice((0, 1, rng.randint(0, 1500))))
                for _ in range(rng.randint(1, 40))]
        block, causal = rng.choice((1, 18, 32, 36, 64, 128, 256)), rng.random() < 0.7
        got = enumerate_items(seqs, block, causal)
        assert sorted(got) == [(b, k) for b, (q, _) in enumerate(seqs) for k in range(-(-q // block))]

        def seen(b, k):
            q, keys = seqs[b]
            vis = min(max(keys - q + min((k + 1) * block, q), 0), keys) if causal else keys
            return -(-vis // 128)
        order = [seen(*x) for x in got]
        assert order == sorted(order, reverse=True)


def test_division_by_multiplication():
    """FastDiv: mul = ceil(2^(31 + bits) / d), exact for every x below 2^31."""
    rng = random.Random(4)
    for d in list(range(1, 300)) + [rng.randrange(1, 1 << 31) for _ in range(300)]:
        bits = (d - 1).bit_length()
        mul, shift = (0, 0) if bits == 0 else (-(-(1 << (31 + bits)) // d), bits - 1)
        assert mul < 1 << 32
        xs = [0, 1, d - 1, d, d + 1, (1 << 31) - 1] + [rng.randrange(1 << 31) for _ in range(50)]
        xs += [k * d + e for k in (1, 2, ((1 << 31) - 1) // d) for e in (-1, 0)]
        for x in xs:
            if 0 <= x < 1 << 31:
                assert (x if d == 1 else ((x * mul) >> 32) >> shift) == x // d
