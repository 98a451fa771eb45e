"""The few-token product's roles when a wait runs out, as a model on the CPU.

The warp that issues the MMAs waits for each buffer of widened codes at a hardware barrier without a
limit; the warps that fill it arrive there. Once a wait has run out (it may be any of the others, at any
time) every role still has to come to its end: no barrier ever holds the arrivals of two buffers' fillings,
and none is left with a waiting warp."""
import pathlib
import random
import re

import pytest

SRC = (pathlib.Path(__file__).parents[1] / "gated_deltanet_linear_build_gb300" / "csrc" / "w4_few.cu").read_text()
BUFFERS = int(re.search(r"kABufs = (\d+)", SRC).group(1))


class Stuck(Exception):
    pass


class Model:
    """Steps 0 .. n - 1 use buffer step % BUFFERS; group g of `turns` fills steps g, g + turns, ...; a group
    is four warps that go on by themselves. One warp issues the MMAs of each step in order."""

    def __init__(self, n, turns, ordered, seed):
        self.n, self.turns, self.ordered = n, turns, ordered
        self.rng = random.Random(seed)
        self.abort = False
        self.given_back = [0] * BUFFERS           # phases of a_empty that are complete
        self.inside = [set() for _ in range(BUFFERS)]      # at the named barrier: five warps, one of them issues
        self.passed = [0] * BUFFERS               # its completed generations

    def arrive(self, b, who):
        if who in self.inside[b]:
            raise Stuck("a warp arrives twice in one generation")
        self.inside[b].add(who)
        if len(self.inside[b]) == 5:
            if "mma" not in self.inside[b]:
                raise Stuck("a generation of arrivals alone")
            self.inside[b].clear()
            self.passed[b] += 1

    def limited(self, ready):
        """A wait that may run out: true once ready, false after an abort or its own limit."""
        while True:
            if ready():
                yield True
                return
            if self.abort or self.rng.random() < 0.002:
                self.abort = True
                yield False
                return
            yield None

    def wait(self, ready):
        while not ready():
            yield None

    def filler(self, group, warp):
        ok = True
        for step in range(group, self.n, self.turns):
            b, use = step % BUFFERS, step // BUFFERS
            place = lambda b=b, use=use: self.given_back[b] >= use  # noqa: E731
            if ok or self.ordered:
                for got in self.limited(place):
                    if got is None:
                        yield
                if not got:
                    ok = False
                    if self.ordered:
                        yield from self.wait(place)
            if ok:                                # codes, which may never come
                for got in self.limited(lambda: self.rng.random() < 0.9):
                    if got is None:
                        yield
                ok = got
            yield
            self.arrive(b, (group, warp))

    def issuer(self):
        for got in self.limited(lambda: self.rng.random() < 0.05):     # x, behind which it may be far
            if got is None:
                yield
        for step in range(self.n):
            b = step % BUFFERS
            generation = self.passed[b]
            self.arrive(b, "mma")
            yield from self.wait(lambda b=b, g=generation: self.passed[b] > g)
            self.given_back[b] += 1               # by the MMAs' end or, where a wait ran out, at once
            yield

    def run(self):
        roles = {(g, w): self.filler(g, w) for g in range(self.turns) for w in range(4)}
        roles["mma"] = self.issuer()
        idle = 0
        while roles:
            key = self.rng.choice(list(roles))
            before = (list(self.passed), list(self.given_back), [len(s) for s in self.inside], self.abort, len(roles))
            try:
                for _ in range(self.rng.choice((1, 1, 5, 40))):        # a warp may be far ahead of others
                    next(roles[key])
            except StopIteration:
                del roles[key]
            after = (list(self.passed), list(self.given_back), [len(s) for s in self.inside], self.abort, len(roles))
            idle = 0 if before != after else idle + 1
            if idle > 20000:
                raise Stuck("no role goes on")


@pytest.mark.parametrize("turns", [2, 3])
def test_every_role_ends_when_a_wait_runs_out(turns):
    aborted = 0
    for seed in range(150):
        m = Model(n=3 + seed % 20, turns=turns, ordered=True, seed=seed)
        m.run()
        aborted += m.abort
    assert aborted > 30


def test_arriving_without_the_place_would_not_end():
    stuck = 0
    for seed in range(150):
        try:
            Model(n=3 + seed % 20, turns=2, ordered=False, seed=seed).run()
        except Stuck:
            stuck += 1
    assert stuck > 10


def test_the_kernel_takes_the_place_before_it_arrives():
    widen = SRC[SRC.index("// ======================= codes to f16"):SRC.index("// ======================= results")]
    assert widen.index("place_wait(place_ready") < widen.index("filled_arrive(filled)")
    issue = SRC[SRC.index("// ======================= MMA ="):SRC.index("// ======================= codes to f16")]
    assert "else if (one)" in issue and "tc::mbar_arrive(a_empty + ab)" in issue
