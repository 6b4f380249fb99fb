"""A CPU model of the tile attention kernel's hand-overs (lq_attn_tile.cu, heads
of 64 and 128), run under random interleavings with roles that stall.

A CTA walks units (two row tiles, or one where the second has no rows) of key
tiles. The planning warp describes tile n in bookkeeping slot n mod 8, once the
loaders have filled tile n - 4 (within a unit that is behind the softmax of
tile n - 8), and, if the slot's old tile n - 8 was the last of its unit, once
both softmax groups are done with that unit (`unit_free`).
The loaders wait until the tile is told and its two ring units (K, then V; 3
or 6 units) are empty, and their copies land later. The MMA thread issues PV of
row tile 0, its next QK, PV of row tile 1, its next QK, or both PVs first
between units; what it issues completes later, in order. A softmax group
arrives on `q_ready` at a unit's start, reads a tile's slot when S is there
and again (the keys kept out of the MMA) when O is there, and arrives on
`unit_free` at the unit's end; a unit without rows for it is free at once.

Checked: what a softmax group reads from a slot is its own tile's, and the run
ends. Planted mistakes: a slot rewritten by the loaders' progress alone, which
orders nothing for a group whose next units have no rows for it; and a wait for
every tile of an earlier unit, whose last PV waits for the next unit's keys.

Where waits may run out at any time (a wait limit of one poll), the CTA ends
without a copy or an MMA of its own in flight: the MMA thread and the loaders see
theirs complete before they leave. Planted mistake: loaders that do so only when a
wait of their own has run out.
"""
import random

import pytest

SLOTS, UNIT_SLOTS = 8, 8


class Model:
    """units: (key tiles, row tiles) of each unit; nu: ring units; gives_up:
    how likely a wait that is looked at runs out; drains: whether the loaders
    see their copies land before they leave, or only after giving up."""

    def __init__(self, units, nu, seed, unit_wait="last tile", gives_up=0.0, drains="always"):
        self.rng = random.Random(seed)
        self.units, self.nu, self.unit_wait, self.gives_up, self.drains = units, nu, unit_wait, gives_up, drains
        self.tiles = [u for u, (n, _) in enumerate(units) for _ in range(n)]
        self.firsts = [i == 0 or self.tiles[i - 1] != u for i, u in enumerate(self.tiles)]
        self.slot = [None] * SLOTS
        self.told = self.done = self.told_units = 0
        self.empty = 0              # ring units whose readers have completed, in order
        self.landed = set()
        self.copies = []            # ring units on their way
        self.mmas = []              # what completing MMAs arrive on, in order
        self.counts = {}            # completed phases by barrier
        self.free = [[0, 0] for _ in units]
        self.issues = []
        self.roles = {"planner": self.planner(), "loader": self.loader(), "mma": self.mma(), "group0": self.softmax(0),
                      "group1": self.softmax(1)}

    def add(self, what):
        self.counts[what] = self.counts.get(what, 0) + 1

    def count(self, what):
        return self.counts.get(what, 0)

    # each role yields the condition that it waits for (None: just a step)
    def planner(self):
        for n, u in enumerate(self.tiles):
            if self.firsts[n]:
                if u >= UNIT_SLOTS:
                    yield lambda u=u: sum(self.free[u - UNIT_SLOTS]) == 2
                self.told_units = u + 1
            if n >= SLOTS // 2:
                yield lambda n=n: self.done >= n - SLOTS // 2 + 1
            if n >= SLOTS and {"last tile": self.firsts[n - SLOTS + 1], "any tile": self.tiles[n - SLOTS] != u, "": False}[self.unit_wait]:
                yield lambda n=n: sum(self.free[self.tiles[n - SLOTS]]) == 2
            self.slot[n % SLOTS] = n
            self.told = n + 1
            yield None

    def loader(self):
        for n in range(len(self.tiles)):
            yield lambda n=n: self.told > n
            for unit in (2 * n, 2 * n + 1):
                yield lambda unit=unit: self.empty >= unit - self.nu + 1
                self.copies.append(unit)
                yield None
            self.done = n + 1

    def mma(self):
        waited = {}

        def next_of(what):
            waited[what] = waited.get(what, 0) + 1
            return lambda k=waited[what]: self.count(what) >= k
        pending = None  # row tiles of the tile whose PV is due
        for n in range(-1, len(self.tiles)):
            more = n + 1 < len(self.tiles)
            nxt, fresh, loaded = None, False, False
            if n >= 0:
                yield lambda n=n: 2 * n + 1 in self.landed
            for s in range(1 if n < 0 else 0, 4):
                if more and not loaded and s > 0:
                    yield lambda n=n: 2 * n + 2 in self.landed
                    nxt, fresh, loaded = self.units[self.tiles[n + 1]][1], self.firsts[n + 1], True
                op = 3 - s if fresh and s in (1, 2) else s
                q = op >> 1
                if op & 1 == 0:
                    if n < 0:
                        continue
                    if q < pending:
                        yield next_of(("p_ready", q))
                        self.mmas.append([("o_full", q)])
                    if q == 1:
                        self.mmas.append(["empty"])
                elif more:
                    if q < nxt:
                        if fresh:
                            yield next_of(("q_ready", q))
                        self.mmas.append([("s_full", q)])
                    if q == 1:
                        self.mmas.append(["empty"])
                yield None
            pending = nxt

    def softmax(self, q):
        base = seen = 0
        for u, (n, row_tiles) in enumerate(self.units):
            yield lambda u=u: self.told_units > u
            if q < row_tiles:
                self.add(("q_ready", q))
                for t in range(base, base + n):
                    seen += 1
                    yield lambda k=seen: self.count(("s_full", q)) >= k
                    self.read(q, t, "keys")
                    yield None
                    self.add(("p_ready", q))
                    yield lambda k=seen: self.count(("o_full", q)) >= k
                    yield None
                    self.read(q, t, "values that are not finite")
            base += n
            yield None
            self.free[u][q] = 1

    def leave(self, role, gave_up):
        """What a role does before it leaves, with waits that do not run out."""
        if role == "mma":
            yield lambda: not self.mmas
        if role == "loader" and (gave_up or self.drains == "always"):
            yield lambda: not self.copies

    def read(self, q, tile, what):
        if self.slot[tile % SLOTS] != tile:
            self.issues.append(f"group {q} reads the {what} of tile {self.slot[tile % SLOTS]} for tile {tile}")

    def run(self):
        rng, waits = self.rng, {r: None for r in self.roles}
        weight = {r: 1.0 for r in self.roles}
        leaving = set()
        for _ in range(200000):
            if not self.roles:
                return "in flight" if self.copies or self.mmas else "end"
            ready = [r for r in self.roles if waits[r] is None or waits[r]()]
            late = [r for r in self.roles if r not in ready and r not in leaving and rng.random() < self.gives_up]
            acts = ready + late + ["copy"] * bool(self.copies) + ["mmas"] * bool(self.mmas)
            if not acts:
                if self.gives_up:
                    continue
                return "deadlock"
            if rng.random() < 0.02:  # another role stalls, or none
                weight = {r: 1.0 for r in self.roles}
                weight[rng.choice(list(self.roles))] = rng.choice([0.002, 0.1, 1.0])
            a = rng.choices(acts, [weight.get(x, 1.0) for x in acts])[0]
            if a == "copy":  # copies land in any order
                self.landed.add(self.copies.pop(rng.randrange(len(self.copies))))
            elif a == "mmas":
                for what in self.mmas.pop(0):
                    if what == "empty":
                        self.empty += 1
                    else:
                        self.add(what)
            else:
                try:
                    if a in late:
                        raise StopIteration
                    waits[a] = next(self.roles[a])
                except StopIteration:
                    if a in leaving:
                        del self.roles[a]
                    else:
                        leaving.add(a)
                        self.roles[a], waits[a] = self.leave(a, a in late), None
        return "too long"


UNITS = {
    "rows 300 of one head": [(3, 2), (4, 1)],
    "long tiles": [(20, 2), (20, 1), (20, 2), (20, 1)],
    "short prompts": [(1, 2), (1, 1)] * 10,
    "one row tile after two": [(5, 2), (12, 1), (2, 2), (9, 1), (9, 1)],
    "two row tiles only": [(7, 2)] * 4,
    "one row tile only": [(3, 1)] * 12,
}


@pytest.mark.parametrize("nu", [3, 6])
@pytest.mark.parametrize("units", UNITS.values(), ids=UNITS.keys())
def test_groups_read_their_own_tiles(units, nu):
    for seed in range(40):
        m = Model(units, nu, seed)
        assert m.run() == "end" and not m.issues, (seed, m.issues[:3])


@pytest.mark.parametrize("nu", [3, 6])
@pytest.mark.parametrize("name,unit_wait", [("long tiles", ""), ("one row tile after two", ""), ("long tiles", "any tile")])
def test_planted_mistakes_are_caught(name, unit_wait, nu):
    models = (Model(UNITS[name], nu, seed, unit_wait) for seed in range(300))
    assert any(m.run() != "end" or m.issues for m in models)


@pytest.mark.parametrize("nu", [3, 6])
@pytest.mark.parametrize("units", [[(1, 1)], [(1, 2)], [(3, 2), (2, 1)], [(9, 2)]], ids=str)
def test_nothing_is_in_flight_when_a_cta_gives_up(units, nu):
    for p in (0.05, 0.5):
        for seed in range(100):
            assert Model(units, nu, seed, gives_up=p).run() == "end", seed


@pytest.mark.parametrize("nu", [3, 6])
def test_loaders_that_leave_their_copies_are_caught(nu):
    assert any(Model([(1, 1)], nu, seed, gives_up=0.5, drains="after giving up").run() == "in flight" for seed in range(100))
