"""The 8-bit attention's waits that run out, restated on the host as
test_paged_giveup_cpu.py does for the bf16 kernel: one completion of a copy or a product
is lost, and every role has to leave, every barrier of a warpgroup to be met by all of
its warps, and nothing may be in flight when the CTA ends.  After a wait gave up the
softmax and the results go through their segment without waiting; each warpgroup leaves
where it takes the next one, all of it if one of its warps has seen the word.  (On the
GPU the case is not provoked: no call makes a wait run out.)"""
import random

import pytest

from test_paged8_pipeline_cpu import plans  # noqa: F401  (a fixture)
from test_paged_giveup_cpu import Cta, Group
from test_paged_pipeline_cpu import Barrier


class Cta8(Cta):
    def __init__(self, pl, segments, rng, lost):
        super().__init__(dict(pl, NP=2, pieces=1), segments, rng, lost)
        n = lambda k, c=1: [Barrier(c) for _ in range(k)]  # noqa: E731
        self.team, self.S = pl["team"], pl["SEGS"]
        self.teams = 2 if pl["stream"] else 1
        self.wgs = self.team * self.teams
        self.c_empty = n(pl["NC"], self.team)
        self.q_full, self.q_empty, self.r_full = n(2, 4), n(2), n(2, 4)
        self.s_full, self.s_empty = n(pl["NS"], 2), n(pl["NS"], self.team)
        self.p_full, self.p_empty, self.l_full = n(2, self.team), n(2), n(2, 4 * self.wgs)
        self.segs = [None] * self.S
        self.seg_full, self.seg_empty = n(self.S), n(self.S, 4 * self.wgs + 3 + 4)
        self.groups = [Group(4) for _ in range(self.wgs + 1)]
        self.active = [rng.randint(1, self.team) for _ in segments]

    # a wait that finds the word set gives up at once
    def wait(self, bar, parity, rounds=1):
        t0 = self.time
        while not bar.passes(parity):
            if self.dead:
                return False
            if self.time - t0 > 4000:
                rounds, t0 = rounds - 1, self.time
                if rounds <= 0:
                    self.dead = True
            yield
        return True

    def take(self, g):
        yield from self.wait(self.seg_full[g % self.S], (g // self.S) % 2)
        s = self.segs[g % self.S]
        yield
        self.seg_empty[g % self.S].arrive()
        return s

    def load_k(self):
        pl, u, g = self.pl, 0, 0
        more = ok = True
        while more and ok:
            more = g < len(self.segments)
            ok = yield from self.wait(self.seg_empty[g % self.S], (g // self.S) % 2 ^ 1)
            if not ok:
                break
            self.segs[g % self.S] = self.segments[g] if more else (0, 0)
            self.seg_full[g % self.S].arrive()
            if not more:
                break
            for _ in range(self.segments[g][0]):
                ok = yield from self.wait(self.c_empty[u % pl["NC"]], (u // pl["NC"]) % 2 ^ 1)
                ok = (yield from self.wait(self.k_empty[u % pl["NK"]], (u // pl["NK"]) % 2 ^ 1)) and ok
                if not ok:
                    break
                self.issue("k", self.k_full[u % pl["NK"]])
                u += 1
            g += 1
        if self.dead:
            yield from self.drain_ring(self.k_full, u)

    def score(self):
        pl, u, g, ok = self.pl, 0, 0, True
        while ok:
            s = yield from self.take(g)
            ok = not self.dead
            if not ok or s[0] == 0:
                break
            ok = yield from self.wait(self.q_full[g % 2], (g // 2) % 2)
            for k in range(s[0]):
                ok = (yield from self.wait(self.k_full[u % pl["NK"]], (u // pl["NK"]) % 2)) and ok
                ok = (yield from self.wait(self.s_empty[u % pl["NS"]], (u // pl["NS"]) % 2 ^ 1)) and ok
                if not ok:
                    break
                self.issue("score", self.s_full[u % pl["NS"]], self.k_empty[u % pl["NK"]], *([self.q_empty[g % 2]] if k == s[0] - 1 else []))
                self.s_full[u % pl["NS"]].arrive()
                u += 1
            g += 1
        if self.dead:
            fin = Barrier(1)
            self.issue("score", fin)
            yield from self.drain(fin, 0)

    def value(self):
        pl, u, g, ok = self.pl, 0, 0, True
        while ok:
            s = yield from self.take(g)
            ok = not self.dead
            if not ok or s[0] == 0:
                break
            ok = yield from self.wait(self.o_empty[g % 2], (g // 2) % 2 ^ 1)
            for k in range(s[0]):
                ok = (yield from self.wait(self.v_full[u % pl["NV"]], (u // pl["NV"]) % 2)) and ok
                ok = (yield from self.wait(self.p_full[u % 2], (u // 2) % 2)) and ok
                if not ok:
                    break
                self.issue("value", self.v_empty[u % pl["NV"]], self.p_empty[u % 2], *([self.o_full[g % 2]] if k == s[0] - 1 else []))
                u += 1
            g += 1
        if self.dead:
            fin = Barrier(1)
            self.issue("value", fin)
            yield from self.drain(fin, 0)

    def softmax(self, warp):
        pl, wg, qd, u, g = self.pl, warp // 4, warp % 4, 0, 0
        group = self.groups[wg]
        while True:
            s = yield from self.take(g)
            out = yield from group.meet(self.dead)
            if out or s[0] == 0:
                return
            yield from self.wait(self.l_empty[g % 2], (g // 2) % 2 ^ 1)
            yield from self.wait(self.r_full[g % 2], (g // 2) % 2)
            fresh = True
            for k in range(s[0]):
                i, u = u, u + 1
                if self.teams == 2 and i % 2 != wg // self.team:
                    continue
                b, empty = i % 2, (i // 2) % 2 ^ 1
                if wg % self.team >= self.active[g]:    # no rows: one warp keeps up
                    if qd == 0:
                        yield from self.wait(self.s_full[i % pl["NS"]], (i // pl["NS"]) % 2)
                        self.s_empty[i % pl["NS"]].arrive()
                        self.c_empty[i % pl["NC"]].arrive()
                        yield from self.wait(self.p_empty[b], empty)
                        self.p_full[b].arrive()
                    continue
                if qd == 0:
                    yield from self.wait(self.s_full[i % pl["NS"]], (i // pl["NS"]) % 2)
                    if self.teams == 1:
                        yield from self.wait(self.p_empty[b], empty)
                yield from group.meet(False)
                move = fresh
                while True:
                    if move:
                        j = i - self.teams
                        if not fresh and qd == 0:
                            yield from self.wait(self.p_empty[j % 2], (j // 2) % 2)
                        yield from group.meet(False)
                        yield from group.meet(False)
                    if self.teams == 2:
                        yield from self.wait(self.p_empty[b], empty)
                    if k >= s[0] - s[1] and wg % self.team == self.active[g] - 1:
                        yield from self.wait(self.v_full[i % pl["NV"]], (i // pl["NV"]) % 2)
                    again = yield from group.meet(not move and self.rng.random() < 0.1)
                    if move or not again:
                        break
                    move = True
                fresh = False
                if qd == 0:
                    self.s_empty[i % pl["NS"]].arrive()
                    self.c_empty[i % pl["NC"]].arrive()
                    self.p_full[b].arrive()
            self.l_full[g % 2].arrive()
            g += 1

    def results(self, warp):
        g, group = -1, self.groups[-1]
        while True:
            yield from self.wait(self.seg_full[(g + 1) % self.S], ((g + 1) // self.S) % 2)
            out = yield from group.meet(self.dead)
            if out:
                return
            more = self.segs[(g + 1) % self.S][0] != 0
            if more:
                yield from self.wait(self.q_empty[(g + 1) % 2], ((g + 1) // 2) % 2 ^ 1)
                yield
                self.q_full[(g + 1) % 2].arrive()
                self.r_full[(g + 1) % 2].arrive()
            if g >= 0:
                if warp == 0:
                    yield from self.wait(self.l_full[g % 2], (g // 2) % 2, rounds=1 + self.segments[g][0] // 8)
                yield from group.meet(False)
                if warp == 0:
                    yield from self.wait(self.o_full[g % 2], (g // 2) % 2)
                yield from group.meet(False)
                self.o_empty[g % 2].arrive()
                self.l_empty[g % 2].arrive()
                self.seg_empty[g % self.S].arrive()
            if not more:
                return
            g += 1

    def run(self):
        live = [self.load_k(), self.load_v(), self.score(), self.value()]
        live += [self.softmax(w) for w in range(4 * self.wgs)] + [self.results(w) for w in range(4)]
        while live:
            self.tick()
            self.rng.shuffle(live)
            for role in list(live):
                if self.rng.random() < 0.7:
                    try:
                        next(role)
                    except StopIteration:
                        live.remove(role)
            assert self.time < 40 * 4000, "a role never leaves: %s" % [r.__name__ for r in live]
        assert not any(self.flight.values()), "copies or products in flight when the CTA ends"
        return self.dead


SHAPES = [(64, 16), (128, 16), (64, 32), (128, 32), (128, 64)]


@pytest.mark.parametrize("hd,rp", SHAPES)
def test_every_role_leaves_when_a_completion_is_lost(plans, hd, rp):  # noqa: F811
    seen = 0
    for seed in range(30):
        rng = random.Random(seed * 10 + rp + hd)
        segments = [(rng.choice([1, 2, 3, 5]), rng.choice([0, 1])) for _ in range(rng.choice([1, 3, 6]))]
        lost = rng.randrange(4 * sum(u for u, _ in segments))
        seen += Cta8(plans[hd, rp], segments, rng, lost).run()
    assert seen >= 18                                  # the last completions of a run nobody waits for


@pytest.mark.parametrize("hd,rp", SHAPES)
def test_nothing_gives_up_when_nothing_is_lost(plans, hd, rp):  # noqa: F811
    for seed in range(15):
        rng = random.Random(seed)
        segments = [(rng.choice([1, 2, 3, 7, 30]), rng.choice([0, 1, 2])) for _ in range(rng.choice([1, 6, 12]))]
        assert not Cta8(plans[hd, rp], segments, rng, None).run()
