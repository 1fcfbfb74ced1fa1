"""Models of the product kernel's mbarrier protocols on the CPU: every role is
a coroutine, a random scheduler interleaves them, copies land when it pleases.
A barrier is the hardware's: a wait names a phase by its parity alone, so it
passes whenever the phase before the current one has that parity.  Each
protocol's earlier form is planted beside the kernel's and must be caught."""
import random

import pytest


class Bar:
    """An mbarrier: arrivals and copies outstanding in the current phase."""

    def __init__(self, count):
        self.count, self.phase, self.left, self.tx = count, 0, count, 0

    def _flip(self):
        if self.left == 0 and self.tx == 0:
            self.phase, self.left = self.phase + 1, self.count

    def arrive(self, copies=0):
        assert self.left > 0, "more arrivals than a phase takes"
        self.left, self.tx = self.left - 1, self.tx + copies
        self._flip()

    def land(self):
        self.tx -= 1
        self._flip()

    def passed(self, parity):
        return (self.phase & 1) != parity


def run(rng, roles, idle=()):
    """Steps the roles in random order until all but the `idle` ones (copy
    engines) have ended.  A role yields None (a step) or a condition to wait
    for.  Now and then a role is left aside for long.  True: all ended."""
    waits = {n: None for n in roles}
    lazy = {n: rng.choice((1.0, 1.0, 0.02)) for n in roles}
    while any(n not in idle for n in roles):
        ready = [n for n in roles if waits[n] is None or waits[n]()]
        if not ready:
            return False
        n = rng.choices(ready, [lazy[i] for i in ready])[0]
        try:
            waits[n] = next(roles[n])
        except StopIteration:
            del roles[n]
    return True


# ------------------------------------------------- fp32 boxes of 32 columns --
def boxes(rng, chunks, ring, everyone):
    """Chunks of 32 columns with a side operand: even chunks of a tile are one
    set of warps' work, odd ones the other's.  everyone: all warps pass every
    phase (wait and arrive); else only a chunk's own set does, as both did
    before.  Returns None, or what went wrong."""
    warps = 2                                     # of a set
    full = [Bar(1) for _ in range(ring)]
    done = [Bar(2 * warps if everyone else warps) for _ in range(ring)]
    slot, wrong, flight = [None] * ring, [], []   # slot: what the memory holds
    order = [c for tile in chunks for c in range(tile)]

    def traffic():
        at = 0
        for i in range(len(order)):
            while at < len(order) and at - i < ring:
                full[at % ring].arrive(1)
                flight.append(at)
                at += 1
                yield None
            yield lambda: done[i % ring].passed(i // ring & 1)
            if slot[i % ring] != ("done", i, warps):
                wrong.append(f"stored {slot[i % ring]} as chunk {i}")
            yield None

    def engine():                                 # loads land in any order
        while True:
            yield lambda: bool(flight)
            i = flight.pop(rng.randrange(len(flight)))
            slot[i % ring] = ("loaded", i, 0)
            full[i % ring].land()

    def warp(set_):
        for i, c in enumerate(order):
            mine = c & 1 == set_
            if not mine and not everyone:
                continue
            yield lambda: full[i % ring].passed(i // ring & 1)
            if mine:
                state, j, n = slot[i % ring] or ("empty", i, 0)
                if j != i or state == "empty":
                    wrong.append(f"chunk {i} worked on {slot[i % ring]}")
                slot[i % ring] = ("done", i, n + 1)
                yield None
            done[i % ring].arrive()

    roles = {"traffic": traffic(), "engine": engine()}
    for s in (0, 1):
        for w in range(warps):
            roles[f"set {s} warp {w}"] = warp(s)
    try:
        if not run(rng, roles, idle=("engine",)) and not wrong:
            wrong.append("nothing can go on")
    except AssertionError as e:
        wrong.append(str(e))
    return wrong[0] if wrong else None


@pytest.mark.parametrize("chunks,ring", [((8,), 3), ((8, 8, 8), 3), ((4,) * 6, 3), ((8, 7, 8, 7), 2),
                                         ((7, 7, 7), 3), ((1, 1, 3, 8), 2)])
def test_boxes_of_half_the_warps(chunks, ring):
    for seed in range(300):
        assert boxes(random.Random(seed), chunks, ring, True) is None, seed


@pytest.mark.parametrize("chunks,ring", [((8,), 3), ((8, 7, 8, 7), 2)])
def test_boxes_whose_other_warps_skip_are_caught(chunks, ring):
    assert any(boxes(random.Random(s), chunks, ring, False) for s in range(300))


# ------------------------------- a pair of CTAs whose shifting warps fill a ring --
def pair(rng, steps, stages, idle_walks):
    """Both operands are shifted: each CTA's shifting warps write a stage, the
    first CTA's tensor cores read both parts and free it in both.  idle_walks: the second CTA's loading warp, which has
    nothing to load, still waits for every stage, as it did before."""
    warps = 2
    full = [Bar(1 + 2 * warps) for _ in range(stages)]
    empty, empty2 = [Bar(1) for _ in range(stages)], [Bar(1) for _ in range(stages)]
    part = [[None] * stages for _ in range(2 * warps)]
    wrong = []

    def walk():
        for i in range(steps):
            yield i, i % stages, i // stages & 1

    def loads(cta):
        for i, s, ph in walk():
            if cta == 0 or idle_walks:
                yield lambda: (empty if cta == 0 else empty2)[s].passed(ph ^ 1)
            if cta == 0:
                full[s].arrive()

    def shifts(cta, w):
        for i, s, ph in walk():
            yield lambda: (empty if cta == 0 else empty2)[s].passed(ph ^ 1)
            part[cta * warps + w][s] = i
            yield None
            full[s].arrive()

    def tensor():
        for i, s, ph in walk():
            yield lambda: full[s].passed(ph)
            if any(p[s] != i for p in part):
                wrong.append(f"step {i} read {[p[s] for p in part]}")
            for e in (empty, empty2):
                yield None
                e[s].arrive()

    roles = {"tensor": tensor(), "loads 0": loads(0), "loads 1": loads(1)}
    for c in (0, 1):
        for w in range(warps):
            roles[f"shift {c} {w}"] = shifts(c, w)
    try:
        if not run(rng, roles):
            wrong.append("waits without end: " + ", ".join(roles))
    except AssertionError as e:
        wrong.append(str(e))
    return wrong[0] if wrong else None


@pytest.mark.parametrize("steps,stages", [(1, 3), (12, 3), (13, 4), (40, 3)])
def test_pair_of_shifting_ctas(steps, stages):
    for seed in range(300):
        assert pair(random.Random(seed), steps, stages, False) is None, seed


def test_pair_whose_idle_loader_walks_is_caught():
    """It can fall two phases behind and wait for one that never comes."""
    bad = [pair(random.Random(s), 12, 3, True) for s in range(2000)]
    assert any(b and "waits without end: loads 1" in b for b in bad)


# ------------------------------------ the loads in flight when a wait gives up --
def drained_too_soon(stages, steps, gave, parity_of):
    """The walk of `steps` stages gave up before step `gave`; the last load of
    every slot is in flight.  Slots whose wait would not stop for it."""
    full = [Bar(1) for _ in range(stages)]
    flight = set()
    for i in range(gave):
        if i % stages in flight:
            full[i % stages].land()          # the tensor cores have taken it
        full[i % stages].arrive(1)
        flight.add(i % stages)
    return [q for q in range(stages) if full[q].passed(parity_of(q, gave, steps, stages)) != (q not in flight)]


def where_it_stopped(q, gave, steps, stages):
    s, ph = gave % stages, gave // stages & 1
    return ph if q < s else ph ^ 1


def where_the_walk_ends(q, gave, steps, stages):     # as it was before
    return steps // stages & 1


def test_drain_waits_for_every_load_in_flight():
    cases = [(st, n, g) for st in (3, 4, 9) for n in range(1, 30) for g in range(n)]
    assert not any(drained_too_soon(*c, where_it_stopped) for c in cases)
    assert any(drained_too_soon(*c, where_the_walk_ends) for c in cases)


# ------------------------------------------ a warp's lanes when a wait gives up --
def lanes_leave(rng, vote, lanes=4, steps=6):
    """Each lane waits for itself, and one may give up at the moment at which
    the barrier completes for another; the loop holds a step that all lanes
    take together.  vote: they agree on going on.  True: all lanes ended."""
    fails = rng.randrange(steps)
    gives_up = [rng.random() < 0.5 for _ in range(lanes)]
    met, votes = [0] * lanes, [[] for _ in range(lanes)]

    def together(i):
        met[i] += 1
        want = met[i]
        return lambda: all(m >= want for m in met)

    def lane(i):
        for s in range(steps):
            live = not (s == fails and gives_up[i])
            if vote:
                votes[i].append(live)
                yield lambda: all(len(v) > s for v in votes)
                live = all(v[s] for v in votes)
            yield together(i)             # a store issued by one elected lane
            if not live:
                return
            yield together(i)             # the next load's

    return run(rng, {i: lane(i) for i in range(lanes)})


def test_lanes_give_up_together():
    assert all(lanes_leave(random.Random(s), True) for s in range(200))
    assert not all(lanes_leave(random.Random(s), False) for s in range(200))
