"""How the kernels on CTA pairs end, replayed on the CPU in random interleavings (no GPU needed).

gemm_kernel (gemm.cuh) and chainn_kernel (chainn.cuh) commit their MMAs to
barriers of both CTAs: each commit of the even CTA's MMA thread becomes an
arrival in either CTA, delivered some time after the MMAs are done, and not in
step with the other CTA's.  Shared memory that an arrival is still on its way to
must not be given up: an arrival at a CTA that has left is an error here.  What
each CTA waits for before the closing cluster barrier has to rule it out: its
epilogue for the last accumulator, and pair_exit (chain_tc.cuh), once the CTA's roles
have ended, for the release of the last ring round's slots and, in the odd CTA, for
the last commit of all (in the even one its MMA thread does).  The waits that the kernels had before, and each of
these left out, are caught.
"""
import pytest

from test_feedforward_protocol_model import Barrier, Broken, World


class Inbox(Barrier):
    """A barrier of a CTA that may have left."""

    def __init__(self, count, cta):
        super().__init__(count)
        self.cta = cta

    def arrive(self):
        if self.cta["left"]:
            raise Broken("an arrival at a CTA that has left")
        super().arrive()


def pair_exit(seed, units, ring, missing=()):
    """units: slots of each unit in turn.  An accumulator a unit, two in turn."""
    w = World(seed)
    ctas = [{"left": False}, {"left": False}]
    full = [Inbox(2, ctas[0]) for _ in range(ring)]
    empty = [[Inbox(1, c) for _ in range(ring)] for c in ctas]
    acc_full = [[Inbox(1, c) for _ in range(2)] for c in ctas]
    acc_empty = [Inbox(2, ctas[0]) for _ in range(2)]
    drain = [Inbox(1, c) for c in ctas]
    copies, tensor = [w.engine(), w.engine()], w.engine()
    panels = [(u, k) for u, n in enumerate(units) for k in range(n)]
    running, ends, at_barrier = [0, 0], [None, None], set()

    def commit(*bars):
        """An arrival at each barrier once the MMAs issued so far are done: on its own from then on."""
        def done():
            for b in bars:
                w.engine().append(b.arrive)
        tensor.append(done)

    def loader(cta):
        slot = phase = uses = 0
        for _ in panels:
            yield (empty[cta][slot], phase ^ 1, uses - 1)
            copies[cta].append(full[slot].arrive)
            slot += 1
            if slot == ring:
                slot, phase, uses = 0, phase ^ 1, uses + 1
        ends[cta] = slot, phase, uses

    def mma():
        for i, (u, k) in enumerate(panels):
            a, slot = u & 1, i % ring
            if k == 0:
                yield (acc_empty[a], (u >> 1 & 1) ^ 1, (u >> 1) - 1)
            yield (full[slot], i // ring & 1, i // ring)
            commit(*(empty[c][slot] for c in range(2)))
            if k + 1 == units[u]:
                commit(*(acc_full[c][a] for c in range(2)))
        commit(*drain)
        yield (drain[0], 0, 0)

    def epilogue(cta):
        for u in range(len(units)):
            yield (acc_full[cta][u & 1], u >> 1 & 1, u >> 1)
            yield True  # (the loads)
            acc_empty[u & 1].arrive()

    def leave(cta):
        """pair_exit: the slots before the loader's next one in this round, the others in the last (without a use: at once)."""
        slot, phase, uses = ends[cta]
        if "releases" not in missing:
            for i in range(ring):
                yield (empty[cta][i], phase, uses) if i < slot else (empty[cta][i], phase ^ 1, uses - 1)
        if cta == 1 and "last commit" not in missing:
            yield (drain[1], 0, 0)

    def role(cta, r):
        running[cta] += 1
        yield from r
        running[cta] -= 1
        if running[cta]:
            return
        yield from leave(cta)  # (this CTA's roles have ended)
        at_barrier.add(cta)
        if len(at_barrier) == 2:  # (the cluster barrier: both CTAs leave)
            for c in ctas:
                c["left"] = True

    w.run([role(*r) for r in ((0, loader(0)), (1, loader(1)), (0, mma()), (0, epilogue(0)), (1, epilogue(1)))])
    assert all(c["left"] for c in ctas)


UNITS = [[1], [1, 1, 1, 1], [7, 2, 5], [16], [3, 1, 1, 9, 4, 4]]


@pytest.mark.parametrize("units", UNITS, ids=str)
@pytest.mark.parametrize("ring", [2, 5, 6])
def test_no_arrival_finds_its_cta_gone(units, ring):
    for seed in range(60):
        pair_exit(seed, units, ring)


@pytest.mark.parametrize("missing", [("releases", "last commit"), ("releases",), ("last commit",)], ids="-".join)
def test_waits_left_out_are_caught(missing):
    caught = 0
    for seed in range(400):
        try:
            pair_exit(seed, [3, 1, 1, 9], 2, missing)
        except Broken as e:
            assert "left" in str(e)
            caught += 1
    assert caught


def gives_up(seed, ring, settle):
    """A wait runs out: the even CTA's loader stops before the odd one's, whose last copies it has not armed its barrier for
    and does not wait for."""
    w = World(seed)
    ctas = [{"left": False}, {"left": False}]
    full = [Inbox(2, ctas[0]) for _ in range(ring)]
    copies = [w.engine(), w.engine()]
    even = w.rng.randint(0, ring - 1)
    running = [0]

    class Landed:
        """The time that pair_exit then waits is more than a copy takes."""

        def ready(self, *_):
            return not copies[1]

    def loader(cta, n):
        yield True
        for i in range(n):
            copies[cta].append(full[i].arrive)
            yield True
        if cta == 0:
            for i in range(n):
                yield (full[i], 0, 0)
        elif settle:
            yield (Landed(), 0, 0)

    def role(r):
        running[0] += 1
        yield from r
        running[0] -= 1
        if not running[0]:
            for c in ctas:
                c["left"] = True

    w.run([role(loader(0, even)), role(loader(1, w.rng.randint(even, ring)))])


def test_copies_of_a_run_that_gave_up_land_before_exit():
    for seed in range(300):
        gives_up(seed, 6, True)
    caught = 0
    for seed in range(300):
        try:
            gives_up(seed, 6, False)
        except Broken:
            caught += 1
    assert caught
