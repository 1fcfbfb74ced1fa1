"""A model of the rounds of a Newton-Schulz tile: two sets of sums, filled in turn
by the products and joined by the epilogue's warps of both CTAs, in any order of
events that the barriers allow."""
import random

import pytest


class Barrier:
    def __init__(self, count):
        self.count, self.have, self.phase = count, 0, 0

    def arrive(self):
        self.have += 1
        assert self.have <= self.count
        if self.have == self.count:
            self.have, self.phase = 0, self.phase ^ 1

    def passed(self, parity):
        return self.phase != parity


class Place:
    """A set in turn and the parity of its barriers."""

    def __init__(self):
        self.set = self.phase = 0

    def next(self):
        self.set ^= 1
        self.phase ^= self.set == 0


def run(seed, early=False):
    """Whether every sum has its rounds.  `early`: the fault of a set given back before it has been read."""
    pick = random.Random(seed)
    rounds = [pick.choice((1, 1, 2, 3, 4, 5)) for _ in range(pick.randint(1, 10))]
    ctas, warps = 2, 3
    full = [[Barrier(1) for _ in range(2)] for _ in range(ctas)]
    empty = [Barrier(ctas * warps) for _ in range(2)]
    holds = [[None, None] for _ in range(ctas)]
    sums = {}

    def products():
        at = Place()
        for tile, n in enumerate(rounds):
            for r in range(n):
                while not empty[at.set].passed(at.phase ^ 1):
                    yield
                for c in range(ctas):
                    holds[c][at.set] = (tile, r)
                yield
                for c in range(ctas):
                    full[c][at.set].arrive()
                at.next()

    def epilogue(cta, warp):
        at = Place()
        for tile, n in enumerate(rounds):
            total = []
            for r in range(1, n):
                before = at.set
                while not full[cta][at.set].passed(at.phase):
                    yield
                at.next()
                while not full[cta][at.set].passed(at.phase):
                    yield
                if early:
                    empty[before].arrive()
                    yield
                total += [holds[cta][before]]
                if not early:
                    empty[before].arrive()
                yield
            while not full[cta][at.set].passed(at.phase):
                yield
            yield
            sums[cta, warp, tile] = total + [holds[cta][at.set]]
            empty[at.set].arrive()
            at.next()

    roles = [products()] + [epilogue(c, w) for c in range(ctas) for w in range(warps)]
    for _ in range(100000):
        if not roles:
            break
        role = pick.choice(roles)
        try:
            next(role)
        except StopIteration:
            roles.remove(role)
    assert not roles, f"stuck: {rounds}"
    return all(sums[c, w, t] == [(t, r) for r in range(n)] for c in range(ctas) for w in range(warps) for t, n in enumerate(rounds))


@pytest.mark.parametrize("seed", range(40))
def test_every_round_is_added_once(seed):
    assert all(run(seed * 100 + i) for i in range(10))


def test_a_set_given_back_early_is_caught():
    assert not all(run(seed, early=True) for seed in range(100))
