"""A model of the 8-bit chunk kernel's barriers, run with random times. What the producer and the converter warps wait for and
arrive on, in which order, and the rings' lengths are read out of the kernel's source; copies, conversions, softmax and
products take times of their own, copies now and then very long ones. A wait by parity passes as the hardware's does: also
when the phase two before the one that is meant is the last complete one. The model records every converter that reads
codes, scales or a place that are not its tile's, every product of parts that are not all there, and a state in which
nobody can go on."""

import heapq
import random
import re

import pytest

import test_kernel_sources_cpu as sources

TEXT = sources.source("paged_chunk8.cu")


def constant(name, d):
    both = re.search(rf"constexpr (?:static )?int {name} = D == 64 \? (\d+) : (\d+)", TEXT)
    if both:
        return int(both.group(1 if d == 64 else 2))
    return int(re.search(rf"constexpr int {name} = (\d+)", TEXT).group(1))


def producer_steps():
    """The producer's steps of one tile, in the order of its source: ("room", -), ("arrive", barrier), ("copy", k or v)."""
    begin = TEXT.index("for (int i = 0; i < tiles; ++i) {")
    body = TEXT[begin:TEXT.index("++piece;", begin)]
    steps = []
    for m in re.finditer(r"\broom\(\d+\)|mbar_arrive\((\w+) \+ n % C::RING\)|copy\(&tm_([kv])", body):
        steps.append(("arrive", m.group(1)) if m.group(1) else ("copy", m.group(2)) if m.group(2) else ("room", None))
    return steps


def end_barriers():
    """The barriers that the producer arrives on for the tile that does not exist, behind the last one."""
    begin = TEXT.index("what = kInfoEnd")
    return re.findall(r"mbar_arrive\((\w+) \+ n % C::RING\)", TEXT[begin:TEXT.index("}", begin)])


def converter_waits():
    """The barriers that a converter waits for before it reads a tile's description: (of keys, of values)."""
    begin = TEXT.index("x += kConverters")
    m = re.search(r"wait\((?:\(value \? (\w+) : (\w+)\)|(\w+)) \+ j % C::RING", TEXT[begin:])
    return (m.group(3), m.group(3)) if m.group(3) else (m.group(2), m.group(1))


class Barrier:
    def __init__(self, count):
        self.count = self.pending = count
        self.phases = 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.phases = self.count, self.phases + 1

    def passes(self, parity):
        return (self.phases & 1) != (parity & 1)


class Model:
    def __init__(self, d, tiles, seed, slow, waits=None):
        self.rng, self.slow, self.tiles, self.errors = random.Random(seed), slow, tiles, []
        self.waits = waits or converter_waits()
        self.nsc, self.ring, self.warps = constant("NSC", d), constant("RING", d), constant("kConverters", d)
        self.n_of = {0: constant("NSK", d), 1: constant("NSV", d)}
        self.ahead = d == 64
        self.c_full = [Barrier(1) for _ in range(self.nsc)]
        self.c_empty = [Barrier(4) for _ in range(self.nsc)]
        self.full = {v: [Barrier(4) for _ in range(n)] for v, n in self.n_of.items()}
        self.empty = {v: [Barrier(1) for _ in range(n)] for v, n in self.n_of.items()}
        self.by_tile = {}
        self.codes = [None] * self.nsc
        self.operand = {v: [dict() for _ in range(n)] for v, n in self.n_of.items()}
        self.info = [None] * self.ring
        self.scores, self.weights = [False] * tiles, [False] * tiles  # whether they are there, by tile
        self.later, self.waiting, self.now = [], [], 0.0

    def named(self, name):
        return self.by_tile.setdefault(name, [Barrier(1) for _ in range(self.ring)])

    def expect(self, good, *what):
        if not good:
            self.errors.append(what)

    def some(self, most):
        return self.rng.random() * most

    # each role yields ("until", condition) or ("after", time)

    def producer(self):
        nc = 0
        steps, ends = producer_steps(), end_barriers()
        for n in range(self.tiles + 1):
            for kind, what in steps if n < self.tiles else [("room", None)] + [("arrive", b) for b in ends]:
                if kind == "room":
                    if nc >= self.nsc:
                        bar, parity = self.c_empty[nc % self.nsc], nc // self.nsc - 1
                        yield "until", lambda: bar.passes(parity)
                elif kind == "arrive":
                    self.info[n % self.ring] = n
                    self.named(what)[n % self.ring].arrive()
                else:
                    st, nc = nc % self.nsc, nc + 1
                    self.codes[st] = None
                    self.start(self.copy(st, (n, int(what == "v"))))
                yield "after", self.some(0.2)

    def copy(self, st, what):
        yield "after", self.some(self.slow if self.rng.random() < 0.1 else 1.0)
        self.codes[st] = what
        self.c_full[st].arrive()

    def converter(self, x):
        while True:
            j, value, part = x >> 3, (x >> 2) & 1, x & 3
            nc = 2 * j + value
            bar = self.named(self.waits[value])[j % self.ring]
            yield "until", lambda: bar.passes(j // self.ring)
            self.expect(self.info[j % self.ring] == j, "description", x, self.info[j % self.ring])
            if j >= self.tiles:
                return
            st, ns, code = j % self.n_of[value], self.n_of[value], nc % self.nsc
            yield "until", lambda: self.c_full[code].passes(nc // self.nsc)
            if j >= ns:
                yield "until", lambda: self.empty[value][st].passes(j // ns - 1)
            for _ in range(2):  # as it begins and as it ends
                self.expect(self.codes[code] == (j, value), "codes", x, self.codes[code])
                self.expect(self.info[j % self.ring] == j, "description", x, self.info[j % self.ring])
                old = self.operand[value][st].get(part, j - ns)
                self.expect(old == j - ns, "place", x, old)
                yield "after", self.some(0.6)
            self.operand[value][st][part] = j
            self.full[value][st].arrive()
            self.c_empty[code].arrive()
            yield "after", self.some(0.1)
            x += self.warps

    def product(self, value, j):
        """The j-th product of keys (scores) or of values: it reads its operand and frees it."""
        st = j % self.n_of[value]
        bar = self.full[value][st]
        yield "until", lambda: bar.passes(j // self.n_of[value])
        if value:
            yield "until", lambda: self.weights[j]
        for _ in range(2):
            self.expect(self.operand[value][st] == dict.fromkeys(range(4), j), "operand", value, j, dict(self.operand[value][st]))
            yield "after", self.some(0.4)
        self.empty[value][st].arrive()
        if not value:
            self.scores[j] = True

    def issuer(self):
        yield from self.product(0, 0)
        for j in range(self.tiles):
            first = [(1, j)] if j + 1 == self.tiles else [(0, j + 1), (1, j)] if self.ahead else [(1, j), (0, j + 1)]
            for value, at in first:
                yield from self.product(value, at)

    def softmax(self):
        for j in range(self.tiles):
            yield "until", lambda: self.scores[j]
            self.expect(self.info[j % self.ring] == j, "description", j, self.info[j % self.ring])
            yield "after", self.some(0.8)
            self.weights[j] = True

    # ---- time

    def start(self, role):
        self.push(role, self.now)

    def push(self, role, when):
        heapq.heappush(self.later, (when, self.rng.random(), role))

    def run(self):
        for role in [self.producer(), self.issuer(), self.softmax(), *(self.converter(x) for x in range(self.warps))]:
            self.start(role)
        while self.later:
            self.now, _, role = heapq.heappop(self.later)
            self.go_on(role)
            moved = True
            while moved:  # whoever waited for what has happened
                moved = False
                for item in list(self.waiting):
                    if item[1]():
                        self.waiting.remove(item)
                        self.push(item[0], self.now + self.some(0.05))
                        moved = True
            if len(self.errors) > 20:
                break
        if self.waiting and not self.errors:
            self.errors.append(("stuck", len(self.waiting)))
        return self.errors

    def go_on(self, role):
        try:
            kind, what = next(role)
        except StopIteration:
            return
        if kind == "after":
            self.push(role, self.now + what)
        elif what():
            self.push(role, self.now)
        else:
            self.waiting.append((role, what))


@pytest.mark.parametrize("slow", [1.0, 10.0, 100.0])
@pytest.mark.parametrize("tiles", [1, 2, 3, 5, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_converters_read_their_own_tile_whatever_the_times(d, tiles, slow):
    for seed in range(40):
        errors = Model(d, tiles, seed, slow).run()
        assert not errors, (seed, errors[:3])


def test_the_model_sees_codes_read_before_they_are_there():
    """Without the wait that says that the stage of a tile's values is free the early reads come back, of values alone."""
    early = [e for seed in range(40) for e in Model(128, 40, seed, 10.0, ("info_full", "info_full")).run() if e[0] == "codes"]
    assert early and all((e[1] >> 2) & 1 for e in early)
