"""The stream schedule of pa_attend, restated in Python integers: closed forms, cuts and parts.

Mirrors AttendWalk (csrc/pa_attend.cuh): every tile of every item belongs to exactly one CTA,
and the parts of a cut item are a run of CTAs, one slot each, as the merge kernel reads them.
"""
import random

import pytest

CHARGE, MIN_SHARE = 320, 320


class Schedule:
    def __init__(self, lens, units, tokens, keys, causal, grid, few=0):
        self.units, self.t, self.keys, self.causal, self.few = units, tokens, keys, causal, few
        self.seqs = [(n, T) for n, T in lens]
        self.items, at = [], 0
        for s, (n, T) in enumerate(self.seqs):
            for u in range(units if n else 0):
                for j in range(self.runs(n)):
                    seen = self.seen(n, T, j)
                    cost = self.cost_of(n, j, seen)
                    self.items.append((s, u, j, -(-seen // keys), at, cost))
                    at += cost
        self.total = at
        self.ctas = max(1, min(grid, at // MIN_SHARE))
        self.snap = max(1, min(at // self.ctas // (16 * keys), 1 << 20))

    def runs(self, n):
        return -(-n // self.t)

    def seen(self, n, T, j):
        return max(T - n + min(n, (j + 1) * self.t), 0) if self.causal else T

    def cost_of(self, n, j, seen):
        return CHARGE + ((seen + 1) // 2 if n - j * self.t <= self.few else seen)

    def before(self, n, T, j):
        every = j > 0 and j * self.t >= n
        full = j - 1 if every else j
        total = full * CHARGE + (self.cost_of(n, j - 1, T) if every else 0)
        if not self.causal:
            return total + full * T
        over = T - n
        i0 = 0 if over >= 0 else min(-over // self.t, full)
        m = full - i0
        return total + m * over + self.t * ((i0 + 1 + full) * m // 2)

    def start(self, c):
        q, r = divmod(self.total, self.ctas)
        return q * c + r * c // self.ctas

    def cut(self, item, x):
        _, _, _, tiles, at, cost = item
        if x <= at:
            return 0
        if x >= at + cost:
            return tiles
        c = (x - at) * tiles // cost
        return 0 if c < self.snap else tiles if tiles - c < self.snap else c


def random_lens(rng):
    kind = rng.choice(["few", "many", "long", "odd"])
    s = {"few": rng.randint(1, 5), "many": rng.randint(20, 80), "long": 1, "odd": rng.randint(1, 20)}[kind]
    out = []
    for _ in range(s):
        n = rng.choice([0, 1, 2, rng.randint(0, 40), rng.randint(0, 900)])
        T = rng.choice([0, 1, n, max(0, n - rng.randint(0, 50)), n + rng.randint(0, 5000), rng.randint(0, 200)])
        if kind == "long":
            n, T = rng.randint(1, 700), rng.randint(20000, 100000)
        out.append((n, T))
    return out


@pytest.mark.parametrize("seed", range(150))
def test_every_tile_once(seed):
    rng = random.Random(seed)
    lens = random_lens(rng)
    tokens = rng.choice([1, 2, 7, 16, 64, 256])
    sch = Schedule(lens, rng.choice([1, 3, 8]), tokens, rng.choice([32, 128]), rng.choice([False, True]),
                   rng.choice([1, 152, 304]), few=rng.choice([0, tokens // 2]))
    for n, T in lens:
        for j in range(sch.runs(n) + 1):
            assert sch.before(n, T, j) == sum(sch.cost_of(n, i, sch.seen(n, T, i)) for i in range(j))
    shares = [(sch.start(c), sch.start(c + 1)) for c in range(sch.ctas)]
    assert shares[0][0] == 0 and shares[-1][1] == sch.total
    for item in sch.items:
        _, _, _, tiles, at, cost = item
        owners = []
        for c, (lo, hi) in enumerate(shares):
            if hi <= at or lo >= at + cost:
                continue
            a, b = sch.cut(item, lo), sch.cut(item, hi)
            if b > a or (tiles == 0 and lo <= at < hi):
                owners.append((c, a, b))
        assert [a for _, a, _ in owners] + [tiles] == [0] + [b for _, _, b in owners]
        assert [c for c, _, _ in owners] == list(range(owners[0][0], owners[0][0] + len(owners)))
        if len(owners) > 1:
            # the second owner's share begins inside the item, and it is the first cut
            cta = owners[1][0]
            assert 0 < sch.cut(item, shares[cta][0]) < tiles and sch.cut(item, shares[cta - 1][0]) == 0
            last = cta
            while sch.cut(item, sch.start(last + 1)) < tiles:
                last += 1
            assert last - cta + 2 == len(owners)
            # at most one first slot and one second slot per CTA
            assert owners[0][1] == 0 and all(a > 0 for _, a, _ in owners[1:])


def test_shares_are_even():
    """Many items: no CTA gets more than its share and a snapped cut."""
    sch = Schedule([(4000, 4000), (300, 9000), (1, 30000)], 8, 64, 128, True, 152)
    load = [0] * sch.ctas
    for item in sch.items:
        for c in range(sch.ctas):
            lo, hi = sch.start(c), sch.start(c + 1)
            if hi > item[4] and lo < item[4] + item[5]:
                load[c] += max(0, sch.cut(item, hi) - sch.cut(item, lo)) * 128
    assert max(load) <= sch.total / sch.ctas * (1 + 2 / 16) + 256
