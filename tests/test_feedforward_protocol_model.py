"""The barrier protocols of the feed-forward kernels, replayed on the CPU in random interleavings (no GPU needed).

Every role of a kernel is a generator that yields what it waits for: a barrier
and the parity that the kernel's code computes.  A barrier counts arrivals and
completes phases; a wait by parity is checked against the phase that it means,
which the model counts on the side: no barrier may get two phases ahead of a
waiter.  Copies and MMAs complete later than they are issued, in order.  Contents
are tags: a panel in a ring slot, a product in an accumulator, scales in their
place; a reader checks that it finds what it came for, a writer that what it
overwrites has been read.  Planted errors are caught.
"""
import random

import pytest


class Broken(AssertionError):
    pass


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0  # phase: completed ones

    def arrive(self):
        self.pending -= 1
        if self.pending < 0:
            raise Broken("an arrival too many in a phase")
        if self.pending == 0:
            self.phase += 1
            self.pending = self.count

    def ready(self, parity, meant):
        """try_wait.parity: the phase of that parity has completed, i.e. the current one has the other parity."""
        if self.phase > meant + 1:
            raise Broken("a barrier is two phases ahead of a waiter")
        done = (self.phase & 1) != parity
        if done != (self.phase > meant):
            raise Broken("a parity means another phase")
        return done


class World:
    """Roles in random turns, and an in-order queue of asynchronous completions for each engine."""

    def __init__(self, seed):
        self.rng, self.actors, self.engines = random.Random(seed), [], []

    def engine(self):
        self.engines.append([])
        return self.engines[-1]

    def run(self, roles):
        waiting = {i: next(r, None) for i, r in enumerate(roles)}
        for _ in range(2_000_000):
            live = [i for i, w in waiting.items() if w is not None]
            able = [i for i in live if waiting[i] is True or waiting[i][0].ready(waiting[i][1], waiting[i][2])]
            busy = [e for e in self.engines if e]
            if not live and not busy:
                return
            if not able and not busy:
                raise Broken("nobody can go on")
            if busy and (not able or self.rng.random() < 0.4):
                self.rng.choice(busy).pop(0)()
            else:
                i = self.rng.choice(able)
                waiting[i] = next(roles[i], None)
        raise Broken("no end")


def pair_kernel(seed, units, ring, e4m3, warps=2, plant=None):
    """gemm_kernel on one pair of CTAs; units: K panels of each unit in turn; `warps` epilogue warps for each CTA."""
    w = World(seed)
    full = [Barrier(2) for _ in range(ring)]              # (arming by the even CTA and both copies: two tokens here)
    empty = [[Barrier(1) for _ in range(ring)] for _ in range(2)]
    acc_full = [[Barrier(3 if e4m3 else 1) for _ in range(2)] for _ in range(2)]
    acc_empty = [Barrier(2 * warps) for _ in range(2)]
    slots = [[None] * ring for _ in range(2)]             # panel in each CTA's slot
    acc, readers = [None, None], [0, 0]
    scales = [[[None] * 3, [None] * 3] for _ in range(2)]  # by CTA and warp
    copies, tensor = [w.engine(), w.engine()], w.engine()
    panels = [(u, k) for u, n in enumerate(units) for k in range(n)]
    products = panels if e4m3 else [(u, n - 1) for u, n in enumerate(units)]
    seen = [[[] for _ in range(warps)] for _ in range(2)]

    def producer(cta):
        slot = phase = uses = 0
        for p in panels:
            yield (empty[cta][slot], phase ^ 1, uses - 1)

            def land(slot=slot, p=p):
                if slots[cta][slot] is not None:
                    raise Broken("a slot overwritten before it was read")
                slots[cta][slot] = p
                full[slot].arrive()
            copies[cta].append(land)
            slot += 1
            if slot == ring:
                slot, phase, uses = 0, phase ^ 1, uses + 1

    def mma():
        slot = phase = a = a_phase = uses = a_uses = 0
        first = True
        for i, p in enumerate(panels):
            last = i + 1 == len(panels) or panels[i + 1][0] != p[0]
            if e4m3 or first:
                if plant != "accumulator not waited for":
                    yield (acc_empty[a], a_phase ^ 1, a_uses - 1)
            yield (full[slot], phase, uses)
            first = False

            def work(slot=slot, a=a, p=p, start=e4m3 or p[1] == 0, done=e4m3 or last):
                if slots[0][slot] != p or slots[1][slot] != p:
                    raise Broken("the MMA reads another panel")
                if start and readers[a]:
                    raise Broken("an accumulator overwritten before it was read")
                if done:
                    acc[a], readers[a] = p, 2 * warps
                for c in range(2):
                    slots[c][slot] = None
                    empty[c][slot].arrive()
                    if done:
                        acc_full[c][a].arrive()
            tensor.append(work)
            slot += 1
            if slot == ring:
                slot, phase, uses = 0, phase ^ 1, uses + 1
            if e4m3 or last:
                a ^= 1
                if a == 0:
                    a_phase, a_uses = a_phase ^ 1, a_uses + 1
                first = True

    def scale(cta, warp):
        place = 0
        for n, p in enumerate(panels):
            behind = 2 if plant == "scales a panel early" else 1
            if n >= behind:
                m = n - behind
                yield (acc_full[cta][m & 1], (m >> 1) & 1, m >> 1)
            else:
                yield True
            old = scales[cta][warp][place]
            if old is not None and old[1]:
                raise Broken("scales overwritten before they were read")
            scales[cta][warp][place] = [p, warps]
            acc_full[cta][n & 1].arrive()
            place = (place + 1) % 3

    def epilogue(cta, warp):
        a = a_phase = a_uses = place = 0
        for p in products:
            yield (acc_full[cta][a], a_phase, a_uses)
            if e4m3:
                for s in scales[cta]:
                    if s[place][0] != p:
                        raise Broken("another panel's scales")
                    s[place][1] -= 1
                place = (place + 1) % 3
            yield True  # (the loads)
            if acc[a] != p:
                raise Broken("another product")
            seen[cta][warp].append(p)
            readers[a] -= 1
            acc_empty[a].arrive()
            if plant == "released twice" and warp == 0:
                acc_empty[a].arrive()
            yield True  # (sums, stores)
            a ^= 1
            if a == 0:
                a_phase, a_uses = a_phase ^ 1, a_uses + 1

    roles = [producer(0), producer(1), mma()]
    roles += [epilogue(c, i) for c in range(2) for i in range(warps)]
    if e4m3:
        roles += [scale(c, i) for c in range(2) for i in range(2)]
    w.run(roles)
    assert all(s == products for c in seen for s in c)


@pytest.mark.parametrize("e4m3", [False, True], ids=["16 bits", "e4m3"])
@pytest.mark.parametrize("units", [[1], [1, 1, 1, 1], [7, 2, 5], [16], [3, 1, 1, 9, 4, 4]], ids=str)
def test_pair_kernel(e4m3, units):
    for seed in range(40):
        pair_kernel(seed, units, 5 if e4m3 else 6, e4m3)


@pytest.mark.parametrize("plant,e4m3", [("accumulator not waited for", False), ("accumulator not waited for", True),
                                        ("scales a panel early", True), ("released twice", False)])
def test_pair_kernel_planted_errors(plant, e4m3):
    caught = 0
    for seed in range(40):
        try:
            pair_kernel(seed, [1, 2, 1, 3, 1, 4, 1, 6], 5, e4m3, plant=plant)
        except Broken:
            caught += 1
    assert caught


def few_rows_kernel(seed, slots_of_k, ring, e4m3, warps=4, plant=None):
    """One CTA of skinny_kernel."""
    w = World(seed)
    full, empty = [Barrier(1) for _ in range(ring)], [Barrier(1) for _ in range(ring)]
    acc_full, acc_empty = [Barrier(1), Barrier(1)], [Barrier(warps), Barrier(warps)]
    slots, acc, readers = [None] * ring, [None, None], [0, 0]
    copies, tensor = w.engine(), w.engine()
    products = list(range(slots_of_k)) if e4m3 else [slots_of_k - 1]
    seen = [[] for _ in range(warps)]

    def producer():
        slot = phase = uses = 0
        for s in range(slots_of_k):
            yield (empty[slot], phase ^ 1, uses - 1)

            def land(slot=slot, s=s):
                if slots[slot] is not None:
                    raise Broken("a slot overwritten before it was read")
                slots[slot] = s
                full[slot].arrive()
            copies.append(land)
            slot += 1
            if slot == ring:
                slot, phase, uses = 0, phase ^ 1, uses + 1

    def mma():
        slot = phase = a = a_phase = uses = a_uses = 0
        for s in range(slots_of_k):
            if e4m3 and plant != "accumulator not waited for":
                yield (acc_empty[a], a_phase ^ 1, a_uses - 1)
            yield (full[slot], phase, uses)
            done = e4m3 or s + 1 == slots_of_k

            def work(slot=slot, a=a, s=s, done=done):
                if slots[slot] != s:
                    raise Broken("the MMA reads another panel")
                if e4m3 and readers[a]:
                    raise Broken("an accumulator overwritten before it was read")
                slots[slot] = None
                empty[slot].arrive()
                if done:
                    acc[a], readers[a] = s, warps
                    acc_full[a].arrive()
            tensor.append(work)
            slot += 1
            if slot == ring:
                slot, phase, uses = 0, phase ^ 1, uses + 1
            if done:
                a ^= 1
                if a == 0:
                    a_phase, a_uses = a_phase ^ 1, a_uses + 1

    def epilogue(warp):
        a = a_phase = a_uses = 0
        for p in products:
            yield (acc_full[a], a_phase, a_uses)
            yield True
            if acc[a] != p:
                raise Broken("another product")
            seen[warp].append(p)
            if e4m3:
                readers[a] -= 1
                acc_empty[a].arrive()
            a ^= 1
            if a == 0:
                a_phase, a_uses = a_phase ^ 1, a_uses + 1
        if any(s is not None for s in slots):
            raise Broken("the sums take the place of a panel that has not been read")

    w.run([producer(), mma()] + [epilogue(i) for i in range(warps)])
    assert all(s == products for s in seen)


@pytest.mark.parametrize("e4m3", [False, True], ids=["16 bits", "e4m3"])
@pytest.mark.parametrize("n", [1, 2, 3, 5, 6, 17])
def test_few_rows_kernel(e4m3, n):
    for seed in range(40):
        few_rows_kernel(seed, n, 3 if e4m3 else 5, e4m3)
        if e4m3:
            few_rows_kernel(seed, n, 4, True, warps=8)


def test_few_rows_kernel_planted_error():
    caught = 0
    for seed in range(40):
        try:
            few_rows_kernel(seed, 12, 3, True, plant="accumulator not waited for")
        except Broken:
            caught += 1
    assert caught
