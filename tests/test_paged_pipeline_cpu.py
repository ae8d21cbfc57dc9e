"""Paged attention's pipeline, restated on the host: every role as a coroutine
over mbarriers with parity waits, run under random schedules.

A parity wait is only sound while the barrier is at most one phase from the one
waited for: waiting for a phase whose predecessor has not completed reads as
done.  The model's wait therefore knows which phase it means, and fails when
the parity test would pass for another one.  It also checks that no buffer is
written while it is in use, that every segment is processed in order, and that
every role ends.  The plans (buffer counts of each head dimension and tile) are
computed as the kernel computes them."""
import random

import pytest

SEGS = 4


def plan(hd, rp):
    stream = rp <= 64
    slot, q, p = 128 * hd * 2, rp * hd * 2, 128 * rp * 2
    nq, np_ = (2 if rp <= 32 else 1), (2 if stream else 1)
    most = 227 * 1024 - (6656 + 64 * rp) - (nq * q + np_ * 2 * p + 2048)
    ns = min(8, most // slot)
    pieces = 2 if rp >= 64 else 1
    piece = slot // pieces
    nk = (most // piece + 2) // 4 if pieces == 2 else ns // 2
    nv = min(8, (most - nk * slot) // piece)
    return dict(stream=stream, NQ=nq, NP=np_, NK=nk, NV=nv, pieces=pieces)


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0     # phase: completed phases

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passes(self, parity):
        """The hardware's test: the phase with this parity has completed."""
        return (self.phase - 1) % 2 == parity


class Model:
    def __init__(self, pl, segments, rng):
        self.pl, self.segments, self.rng = pl, segments, rng
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
        self.segs = [None] * SEGS
        self.buf = {}                                             # buffer -> what it holds
        self.pending = []                                         # asynchronous work in issue order, per queue
        self.done_results = []
        self.refs = {}

    # wait for the k-th completion (k from 0) of a barrier
    def wait(self, bar, k):
        parity = k % 2
        while not bar.passes(parity):
            assert bar.phase <= k + 1
            yield
        assert bar.phase == k + 1, "the parity test passed for another phase"

    # wait for a buffer to be free for its use number k (from 0): the (k-1)-th completion of its empty barrier
    def free(self, bar, k):
        if k == 0:
            assert bar.passes(1) and bar.phase == 0
            return
        yield from self.wait(bar, k - 1)

    def take(self, g):
        yield from self.wait(self.seg_full[g % SEGS], g // SEGS)
        s = self.segs[g % SEGS]
        assert s is None or s[0] == g
        self.seg_empty[g % SEGS].arrive()
        return s

    def put(self, key, value, must_be=None):
        self.buf[key] = value

    def async_(self, queue, fn):
        self.pending.append((queue, fn))

    # ---- roles ----
    def load_k(self):
        u = 0
        for g in range(len(self.segments) + 1):
            yield from self.free(self.seg_empty[g % SEGS], g // SEGS)
            self.segs[g % SEGS] = (g, self.segments[g]) if g < len(self.segments) else None
            self.seg_full[g % SEGS].arrive()
            if g == len(self.segments):
                return
            nq = self.pl["NQ"]
            yield from self.free(self.q_empty[g % nq], g // nq)
            self.async_("tma", lambda g=g, nq=nq: (self.put(("q", g % nq), g), self.q_full[g % nq].arrive()))
            for _ in range(self.segments[g][0]):
                nk = self.pl["NK"]
                yield from self.free(self.k_empty[u % nk], u // nk)
                self.async_("tma", lambda u=u, nk=nk: (self.put(("k", u % nk), u), self.k_full[u % nk].arrive()))
                u += 1
                yield

    def load_v(self):
        x = 0
        for g in range(len(self.segments) + 1):
            s = yield from self.take(g)
            if s is None:
                return
            for _ in range(s[1][0] * self.pl["pieces"]):
                nv = self.pl["NV"]
                yield from self.free(self.v_empty[x % nv], x // nv)
                self.async_("tmav", lambda x=x, nv=nv: (self.put(("v", x % nv), x), self.v_full[x % nv].arrive()))
                x += 1
                yield

    def score(self):
        u = 0
        for g in range(len(self.segments) + 1):
            s = yield from self.take(g)
            if s is None:
                return
            nq, nk = self.pl["NQ"], self.pl["NK"]
            yield from self.wait(self.q_full[g % nq], g // nq)
            for k in range(s[1][0]):
                yield from self.wait(self.k_full[u % nk], u // nk)
                yield from self.free(self.s_empty[u % 2], u // 2)
                last = k == s[1][0] - 1

                def mma(u=u, g=g, last=last):
                    assert self.buf[("k", u % nk)] == u and self.buf[("q", g % nq)] == g
                    self.put(("s", u % 2), u)
                    self.s_full[u % 2].arrive()
                    self.k_empty[u % nk].arrive()
                    if last:
                        self.q_empty[g % nq].arrive()
                self.async_("score", mma)
                u += 1
                yield

    def value(self):
        u = 0
        pieces, nv, np_ = self.pl["pieces"], self.pl["NV"], self.pl["NP"]
        for g in range(len(self.segments) + 1):
            s = yield from self.take(g)
            if s is None:
                return
            yield from self.free(self.o_empty[g % 2], g // 2)
            for k in range(s[1][0]):
                yield from self.wait(self.p_full[u % np_], u // np_)
                for v in range(pieces):
                    x = u * pieces + v
                    yield from self.wait(self.v_full[x % nv], x // nv)

                    def mma(u=u, x=x, last=v == pieces - 1, end=k == s[1][0] - 1, g=g):
                        assert self.buf[("v", x % nv)] == x and self.buf[("p", u % np_)] == {u}
                        self.v_empty[x % nv].arrive()
                        if last:
                            self.p_empty[u % np_].arrive()
                            if end:
                                self.o_full[g % 2].arrive()
                    self.async_("value", mma)
                    yield
                u += 1

    def softmax(self, warp):
        wg = warp // 4
        u = 0
        pieces, nv, np_ = self.pl["pieces"], self.pl["NV"], self.pl["NP"]
        for g in range(len(self.segments) + 1):
            s = yield from self.take(g)
            if s is None:
                return
            yield from self.free(self.l_empty[g % 2], g // 2)
            for k in range(s[1][0]):
                i, u = u, u + 1
                if self.pl["stream"] and i % 2 != wg:
                    continue
                yield from self.wait(self.s_full[i % 2], i // 2)
                assert self.buf[("s", i % 2)] == i
                yield
                self.s_empty[i % 2].arrive()
                b, use = (i % 2, i // 2) if self.pl["stream"] else (0, i)
                yield from self.free(self.p_empty[b], use)
                held = self.buf.setdefault(("p", b), set())
                if held != {i}:
                    self.buf[("p", b)] = {i}
                masked = k >= s[1][0] - s[1][1]
                if masked and (self.pl["stream"] or wg == 0):
                    for v in range(pieces):
                        x = i * pieces + v
                        yield from self.wait(self.v_full[x % nv], x // nv)
                        assert self.buf[("v", x % nv)] == x
                yield
                self.p_full[b].arrive()
            self.refs[(g % 2, warp)] = g
            yield
            self.l_full[g % 2].arrive()

    def results(self, warp):
        for g in range(len(self.segments) + 1):
            s = yield from self.take(g)
            if s is None:
                return
            yield from self.wait(self.l_full[g % 2], g // 2)
            assert all(self.refs[(g % 2, w)] == g for w in range(8))
            yield
            yield from self.wait(self.o_full[g % 2], g // 2)
            yield
            assert all(self.refs[(g % 2, w)] == g for w in range(8))
            self.o_empty[g % 2].arrive()
            self.l_empty[g % 2].arrive()
            if warp == 0:
                self.done_results.append(g)

    def run(self):
        roles = [self.load_k(), self.load_v(), self.score(), self.value()]
        roles += [self.softmax(w) for w in range(8)] + [self.results(w) for w in range(4)]
        live = dict(enumerate(roles))
        slow = self.rng.choice(list(live) + [None, None])        # one role that lags
        lagging = self.rng.choice(["tma", "tmav", "tk", "tv", "score", "value"])   # one kind of work that lags
        idle = 0
        while live:
            if self.pending and self.rng.random() < 0.4:          # the front of one queue completes
                queue = self.rng.choice(sorted({q for q, _ in self.pending}))
                if queue != lagging or self.rng.random() < 0.01:
                    at = next(i for i, (q, _) in enumerate(self.pending) if q == queue)
                    self.pending.pop(at)[1]()
            r = self.rng.choice(list(live))
            if r == slow and self.rng.random() < 0.9 and len(live) > 1 and idle < 4000:
                idle += 1
                continue
            try:
                next(live[r])
            except StopIteration:
                del live[r]
            idle += 1
            assert idle < 200000, "deadlock"
        while self.pending:
            self.pending.pop(0)[1]()
        assert self.done_results == list(range(len(self.segments)))


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rp", [16, 32, 64, 128])
def test_pipeline_has_no_wrong_phase_no_overwrite_and_no_deadlock(hd, rp):
    pl = plan(hd, rp)
    assert pl["NK"] >= 1 and pl["NV"] >= pl["pieces"] + 1
    for seed in range(60):
        rng = random.Random(seed * 100 + rp + hd)
        # (units, masked units at the end) of each segment
        segments = [(rng.choice([1, 1, 2, 3, 7, 20]), rng.choice([0, 1, 2])) for _ in range(rng.choice([1, 2, 6, 12]))]
        Model(pl, segments, rng).run()


def test_the_model_rejects_slots_shared_by_two_waiters():
    """K and V taking turns in an odd ring (each waited for by another role) is the
    mistake the separate rings avoid: the model has to see it."""
    pl = plan(128, 32)

    class Shared(Model):
        def __init__(self, *a):
            super().__init__(*a)
            n = 5
            full, empty = [Barrier(1) for _ in range(n)], [Barrier(1) for _ in range(n)]
            self.ring = (full, empty, n)

        def load_k(self):
            full, empty, n = self.ring
            f = 0
            for g in range(len(self.segments) + 1):
                yield from self.free(self.seg_empty[g % SEGS], g // SEGS)
                self.segs[g % SEGS] = (g, self.segments[g]) if g < len(self.segments) else None
                self.seg_full[g % SEGS].arrive()
                if g == len(self.segments):
                    return
                nq = self.pl["NQ"]
                yield from self.free(self.q_empty[g % nq], g // nq)
                self.async_("tma", lambda g=g, nq=nq: (self.put(("q", g % nq), g), self.q_full[g % nq].arrive()))
                for _ in range(self.segments[g][0]):
                    for kind in "kv":
                        yield from self.free(empty[f % n], f // n)
                        # copies may land in any order: K in one queue, V in another
                        self.async_("t" + kind, lambda f=f, kind=kind: (self.put(("slot", f % n), (kind, f // 2)), full[f % n].arrive()))
                        f += 1

        def load_v(self):
            for g in range(len(self.segments) + 1):
                s = yield from self.take(g)
                if s is None:
                    return

        def score(self):
            full, empty, n = self.ring
            u = 0
            for g in range(len(self.segments) + 1):
                s = yield from self.take(g)
                if s is None:
                    return
                for k in range(s[1][0]):
                    f = 2 * u
                    yield from self.wait(full[f % n], f // n)
                    yield from self.free(self.s_empty[u % 2], u // 2)
                    last = k == s[1][0] - 1
                    self.async_("score", lambda u=u, f=f, g=g, last=last: (
                        self.put(("s", u % 2), u), self.s_full[u % 2].arrive(), empty[f % n].arrive(),
                        self.q_empty[g % self.pl["NQ"]].arrive() if last else None))
                    u += 1
                    yield

        def value(self):
            full, empty, n = self.ring
            u = 0
            for g in range(len(self.segments) + 1):
                s = yield from self.take(g)
                if s is None:
                    return
                yield from self.free(self.o_empty[g % 2], g // 2)
                for k in range(s[1][0]):
                    b, f = u % self.pl["NP"], 2 * u + 1
                    yield from self.wait(self.p_full[b], u // self.pl["NP"])
                    yield from self.wait(full[f % n], f // n)
                    end = k == s[1][0] - 1
                    self.async_("value", lambda f=f, b=b, g=g, end=end: (
                        empty[f % n].arrive(), self.p_empty[b].arrive(), self.o_full[g % 2].arrive() if end else None))
                    u += 1
                    yield

    wrong = 0
    for seed in range(60):
        try:
            Shared(pl, [(10, 0)], random.Random(seed)).run()
        except AssertionError as e:
            assert "another phase" in str(e), e
            wrong += 1
    assert wrong > 0
