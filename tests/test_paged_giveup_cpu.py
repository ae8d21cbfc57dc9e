"""Paged attention's waits that run out, restated on the host: the roles as
coroutines with waits bounded in time, while one completion of a copy or a
product is lost.  Every role has to leave, every barrier of a warpgroup to be
met by all of its warps, and nothing may be in flight when the CTA ends.  (On
the GPU the case is not provoked: no call makes a wait run out.)"""
import random

import pytest

from test_paged_pipeline_cpu import SEGS, Barrier, plan

LIMIT, LATENCY = 4000, 60          # steps until a wait gives up; until a copy or product completes


class Group:
    """A warpgroup's named barrier: returns to all when all have come, with the OR of their votes."""

    def __init__(self, n):
        self.n, self.round, self.votes, self.result = n, 0, [], False

    def meet(self, vote):
        mine = self.round
        self.votes.append(vote)
        if len(self.votes) == self.n:
            self.result, self.votes, self.round = any(self.votes), [], mine + 1
        while self.round == mine:
            yield
        return self.result


class Cta:
    def __init__(self, pl, segments, rng, lost):
        self.pl, self.segments, self.rng, self.lost = pl, segments, rng, lost
        n = lambda k, c=1: [Barrier(c) for _ in range(k)]
        arrive = 4 if pl["stream"] else 8
        self.k_full, self.k_empty = n(pl["NK"]), n(pl["NK"])
        self.v_full, self.v_empty = n(pl["NV"]), n(pl["NV"])
        self.q_full, self.q_empty = n(pl["NQ"]), n(pl["NQ"])
        self.s_full, self.s_empty = n(2), n(2, arrive)
        self.p_full, self.p_empty = n(pl["NP"], arrive), n(pl["NP"])
        self.o_full, self.o_empty = n(2), n(2, 4)
        self.l_full, self.l_empty = n(2, 8), n(2, 4)
        self.seg_full, self.seg_empty = n(SEGS), n(SEGS, 15)
        self.segs, self.time, self.dead = [None] * SEGS, 0, False
        self.groups = [Group(4), Group(4), Group(4)]
        self.flight = {q: [] for q in ("k", "v", "score", "value")}     # in order: (due, completions)
        self.count = 0

    # ---- time, copies, products ----
    def issue(self, queue, *arrivals):
        """A completion: lost altogether for the chosen one (its data has landed, its signal has not)."""
        me, self.count = self.count, self.count + 1
        due = self.time + self.rng.randint(1, LATENCY)
        self.flight[queue].append((due, () if me == self.lost else arrivals))

    def tick(self):
        self.time += 1
        for q in self.flight.values():
            while q and q[0][0] <= self.time:
                for bar in q.pop(0)[1]:
                    bar.arrive()

    def wait(self, bar, parity, rounds=1):
        t0 = self.time
        while not bar.passes(parity):
            if self.time - t0 > LIMIT:
                if rounds > 1 and not self.dead:
                    rounds, t0 = rounds - 1, self.time
                    continue
                self.dead = True
                return False
            yield
        return True

    def drain(self, bar, parity):
        t0 = self.time
        while not bar.passes(parity) and self.time - t0 < LIMIT:
            yield

    def take(self, g):
        yield from self.wait(self.seg_full[g % SEGS], (g // SEGS) % 2)
        s = self.segs[g % SEGS]
        yield
        self.seg_empty[g % SEGS].arrive()
        return s

    # ---- roles ----
    def load_k(self):
        pl, u, g, ok = self.pl, 0, 0, True
        q = 0
        while ok:
            more = g < len(self.segments)
            ok = yield from self.wait(self.seg_empty[g % SEGS], (g // SEGS) % 2 ^ 1)
            if not ok:
                break
            self.segs[g % SEGS] = self.segments[g] if more else (0, 0)
            self.seg_full[g % SEGS].arrive()
            if not more:
                break
            ok = yield from self.wait(self.q_empty[g % pl["NQ"]], (g // pl["NQ"]) % 2 ^ 1)
            if not ok:
                break
            self.issue("k", self.q_full[g % pl["NQ"]])
            q += 1
            for _ in range(self.segments[g][0]):
                ok = yield from self.wait(self.k_empty[u % pl["NK"]], (u // pl["NK"]) % 2 ^ 1)
                if not ok:
                    break
                self.issue("k", self.k_full[u % pl["NK"]])
                u += 1
            g += 1
        if self.dead:
            yield from self.drain_ring(self.k_full, u)
            yield from self.drain_ring(self.q_full, q)

    def drain_ring(self, bars, used):
        at, rnd = used % len(bars), (used // len(bars)) % 2
        for i, bar in enumerate(bars):
            yield from self.drain(bar, rnd if i < at else rnd ^ 1)

    def load_v(self):
        pl, x, g, ok = self.pl, 0, 0, True
        while True:
            s = yield from self.take(g)
            ok = not self.dead
            if not ok or s[0] == 0:
                break
            for _ in range(s[0] * pl["pieces"]):
                ok = yield from self.wait(self.v_empty[x % pl["NV"]], (x // pl["NV"]) % 2 ^ 1)
                if not ok:
                    break
                self.issue("v", self.v_full[x % pl["NV"]])
                x += 1
            if not ok:
                break
            g += 1
        if self.dead:
            yield from self.drain_ring(self.v_full, x)

    def score(self):
        pl, u, g, ok = self.pl, 0, 0, True
        while ok:
            s = yield from self.take(g)
            ok = not self.dead
            if not ok or s[0] == 0:
                break
            ok = yield from self.wait(self.q_full[g % pl["NQ"]], (g // pl["NQ"]) % 2)
            for _ in range(s[0]):
                ok = ok and (yield from self.wait(self.k_full[u % pl["NK"]], (u // pl["NK"]) % 2))
                ok = ok and (yield from self.wait(self.s_empty[u % 2], (u // 2) % 2 ^ 1))
                if not ok:
                    break
                self.issue("score", self.s_full[u % 2], self.k_empty[u % pl["NK"]])
                u += 1
            if ok:
                self.issue("score", self.q_empty[g % pl["NQ"]])
            g += 1
        if not ok or self.dead:
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
            for _ in range(s[0]):
                if not ok:
                    break
                ok = yield from self.wait(self.p_full[u % pl["NP"]], (u // pl["NP"]) % 2)
                for v in range(pl["pieces"]):
                    x = u * pl["pieces"] + v
                    ok = ok and (yield from self.wait(self.v_full[x % pl["NV"]], (x // pl["NV"]) % 2))
                    if not ok:
                        break
                    self.issue("value", self.v_empty[x % pl["NV"]])
                if not ok:
                    break
                self.issue("value", self.p_empty[u % pl["NP"]])
                u += 1
            if ok:
                self.issue("value", self.o_full[g % 2])
            g += 1
        if not ok or self.dead:
            fin = Barrier(1)
            self.issue("value", fin)
            yield from self.drain(fin, 0)

    def softmax(self, warp):
        pl, wg, u, g, ok = self.pl, warp // 4, 0, 0, True
        group = self.groups[wg]
        while True:
            s = yield from self.take(g)
            out = yield from group.meet(self.dead)
            if out or s[0] == 0:
                return
            ok = ok and (yield from self.wait(self.l_empty[g % 2], (g // 2) % 2 ^ 1))
            for k in range(s[0]):
                i, u = u, u + 1
                if pl["stream"] and i % 2 != wg:
                    continue
                ok = ok and (yield from self.wait(self.s_full[i % 2], (i // 2) % 2))
                yield from group.meet(False)           # references, or whether they move
                yield
                self.s_empty[i % 2].arrive()
                b, use = (i % 2, i // 2) if pl["stream"] else (0, i)
                ok = ok and (yield from self.wait(self.p_empty[b], use % 2 ^ 1))
                if k >= s[0] - s[1] and (pl["stream"] or wg == 0):
                    for v in range(pl["pieces"]):
                        x = i * pl["pieces"] + v
                        ok = ok and (yield from self.wait(self.v_full[x % pl["NV"]], (x // pl["NV"]) % 2))
                self.p_full[b].arrive()
            self.l_full[g % 2].arrive()
            g += 1

    def results(self, warp):
        g = 0
        while True:
            s = yield from self.take(g)
            out = yield from self.groups[2].meet(self.dead)
            if out or s[0] == 0:
                return
            ok = yield from self.wait(self.l_full[g % 2], (g // 2) % 2, rounds=1 + s[0] // 8)
            yield from self.groups[2].meet(False)
            ok = ok and (yield from self.wait(self.o_full[g % 2], (g // 2) % 2))
            yield
            self.o_empty[g % 2].arrive()
            self.l_empty[g % 2].arrive()
            g += 1

    def run(self):
        live = [self.load_k(), self.load_v(), self.score(), self.value()]
        live += [self.softmax(w) for w in range(8)] + [self.results(w) for w in range(4)]
        ends = {}
        bound = 40 * LIMIT
        while live:
            self.tick()
            self.rng.shuffle(live)
            for role in list(live):
                if self.rng.random() < 0.7:
                    try:
                        next(role)
                    except StopIteration:
                        ends[role] = self.time
                        live.remove(role)
            assert self.time < bound, "a role never leaves: %s" % [r.__name__ for r in live]
        assert not any(self.flight.values()), "copies or products in flight when the CTA ends"
        return self.dead


@pytest.mark.parametrize("hd,rp", [(128, 16), (64, 32), (128, 64), (64, 128), (128, 128)])
def test_every_role_leaves_when_a_completion_is_lost(hd, rp):
    pl = plan(hd, rp)
    seen = 0
    for seed in range(40):
        rng = random.Random(seed * 10 + rp + hd)
        segments = [(rng.choice([1, 2, 3, 5]), rng.choice([0, 1])) for _ in range(rng.choice([1, 3, 6]))]
        total = sum(u for u, _ in segments)
        lost = rng.randrange(total * (2 + 2 * pl["pieces"]))
        seen += Cta(pl, segments, rng, lost).run()
    assert seen >= 25                                  # the last completions of a run nobody waits for


@pytest.mark.parametrize("hd,rp", [(128, 16), (64, 32), (128, 64), (64, 128), (128, 128)])
def test_nothing_gives_up_when_nothing_is_lost(hd, rp):
    pl = plan(hd, rp)
    for seed in range(20):
        rng = random.Random(seed)
        segments = [(rng.choice([1, 2, 3, 7, 30]), rng.choice([0, 1, 2])) for _ in range(rng.choice([1, 6]))]
        assert not Cta(pl, segments, rng, None).run()
