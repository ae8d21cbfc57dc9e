"""The 8-bit attention's pipeline on the host: its shared-memory plan, compiled from
the kernel's own header, and its roles as coroutines under random schedules, as
test_paged_pipeline_cpu.py runs the bf16 kernel's.

What is new against that model: the results' warps split the next segment's queries
before they write a segment's results (q_full, and r_full for what the softmax needs
of the rows) and let a segment's entry in the list go when its results are written,
scales arrive with K but have a ring of their own, which a chunk's warpgroups free with
its S^T."""
import os
import random
import subprocess

import pytest

from test_paged_pipeline_cpu import Barrier, Model

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = r"""
#include <stdio.h>
#include "paged_plan8.h"
using namespace sv::plan8;
template <int HD, int RP> void line() {
    using L = Plan<HD, RP>;
    printf("%d %d %d %d %d %d %d %d %d %d %d %d\n", HD, RP, (int)sizeof(Fixed<RP>), L::kBytes, L::NK, L::NV, kScaleSlots, L::kTeam, (int)L::kStream, L::NS, L::kUsed, kSegs);
}
int main() {
    line<64, 16>(); line<64, 32>(); line<64, 64>();
    line<128, 16>(); line<128, 32>(); line<128, 64>();
}
"""
NAMES = ["HD", "RP", "fixed", "bytes", "NK", "NV", "NC", "team", "stream", "NS", "columns", "SEGS"]


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan8")
    (d / "plan.cpp").write_text(SRC)
    inc = os.path.join(ROOT, "speculative_decoding_verify_pass_gb300", "csrc")
    subprocess.check_call(["g++", "-std=c++17", "-I", inc, str(d / "plan.cpp"), "-o", str(d / "plan")])
    rows = [dict(zip(NAMES, map(int, x.split()))) for x in subprocess.check_output([str(d / "plan")]).decode().split("\n") if x]
    return {(r["HD"], r["RP"]): dict(r, pieces=1, NQ=2, NP=2) for r in rows}


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rp", [16, 32, 64])
def test_static_memory_and_tiles_fit(plans, hd, rp):
    r = plans[hd, rp]
    assert r["fixed"] + r["bytes"] <= 227 * 1024 and r["columns"] <= 512
    # K, V, both parts of the queries, three parts of P^T, up to 1 KB of alignment and 1 KB behind the last V
    chunk = 128 * hd
    assert r["bytes"] >= (r["NK"] + r["NV"]) * chunk + 2 * 2 * rp * hd + 2 * 3 * 128 * rp + 2048
    groups = 2 if r["stream"] else 1
    # scales of 8 chunks; per row: references and four sums of two parities and up to two teams, shrinkage, powers of two, weights, token
    assert r["fixed"] >= 8 * 256 + rp * (2 * groups * 5 * 4 + groups * 4 + 2 * 4 + 2 * 8 + 4) + 4 * 1025
    # a slot of scales is always read by the same team (it then sees every phase of its barrier)
    assert r["NC"] % 2 == 0 and r["team"] * groups == (2 if rp == 16 else 4)


class Model8(Model):
    """Softmax warpgroups in two teams that take alternate chunks (a stream), or in one team
    that takes all.  Of a team, warpgroups without rows in a segment only keep up
    with the barriers (absent: they do not, and the first arrives for them).  Of the warp
    that keeps up, one lane arrives: it and the other lanes leave a wait apart, and join
    before it arrives (apart: they do not)."""
    absent = False
    apart = False

    def __init__(self, pl, segments, rng):
        super().__init__(pl, segments, rng)
        n = lambda k, c=1: [Barrier(c) for _ in range(k)]  # noqa: E731
        team = pl["team"]
        self.q_full, self.r_full = n(2, 4), n(2, 4)
        self.c_empty = n(pl["NC"], team)
        self.s_full, self.s_empty = n(pl["NS"], 2), n(pl["NS"], team)
        self.groups = team * (2 if pl["stream"] else 1)
        self.p_full, self.l_full = n(2, team), n(2, 4 * self.groups)
        self.segs = [None] * pl["SEGS"]
        self.seg_full, self.seg_empty = n(pl["SEGS"]), n(pl["SEGS"], 4 * self.groups + 3 + 4)
        self.active = [rng.randint(1, team) for _ in segments]
        self.place = [-1] * self.groups                           # segment of each warpgroup
        self.passed = [[0, 0] for _ in range(self.groups)]        # waits that the arriving lane and the others have left

    def listed(self, g):
        """The list's entry g, not let go yet."""
        n = self.pl["SEGS"]
        yield from self.wait(self.seg_full[g % n], g // n)
        s = self.segs[g % n]
        assert s is None or s[0] == g
        return s

    def take(self, g):
        s = yield from self.listed(g)
        self.seg_empty[g % self.pl["SEGS"]].arrive()
        return s

    def take4(self, g):
        """A warpgroup's four warps take a segment."""
        s = None
        for _ in range(4):
            s = yield from self.take(g)
        return s

    def load_k(self):
        u, nk, nc = 0, self.pl["NK"], self.pl["NC"]
        for g in range(len(self.segments) + 1):
            n = self.pl["SEGS"]
            yield from self.free(self.seg_empty[g % n], g // n)
            self.segs[g % n] = (g, self.segments[g]) if g < len(self.segments) else None
            self.seg_full[g % n].arrive()
            if g == len(self.segments):
                return
            for _ in range(self.segments[g][0]):
                yield from self.free(self.c_empty[u % nc], u // nc)
                yield from self.free(self.k_empty[u % nk], u // nk)
                self.async_("tk", lambda u=u: (self.put(("c", u % nc), u), self.put(("k", u % nk), u), self.k_full[u % nk].arrive()))
                u += 1
                yield

    def score(self):
        u, nk, ns = 0, self.pl["NK"], self.pl["NS"]
        for g in range(len(self.segments) + 1):
            s = yield from self.take(g)
            if s is None:
                return
            yield from self.wait(self.q_full[g % 2], g // 2)
            for k in range(s[1][0]):
                yield from self.wait(self.k_full[u % nk], u // nk)
                yield from self.free(self.s_empty[u % ns], u // ns)

                def mma(u=u, g=g, last=k == s[1][0] - 1):
                    assert self.buf[("k", u % nk)] == u and self.buf[("q", g % 2)] == g
                    self.put(("s", u % ns), u)
                    self.s_full[u % ns].arrive()
                    self.k_empty[u % nk].arrive()
                    if last:
                        self.q_empty[g % 2].arrive()
                self.async_("score", mma)
                self.s_full[u % ns].arrive()
                u += 1
                yield

    def join(self, wg, lane):
        """The warp that keeps up leaves a wait: its arriving lane (0), the others (1)."""
        n = self.passed[wg]
        n[lane] += 1
        while not self.apart and n[1 - lane] < n[lane]:
            yield

    def other_lanes(self, wg):
        """Of the warp that keeps up while its warpgroup has no rows."""
        u, ns, team = 0, self.pl["NS"], self.pl["team"]
        for g, (units, _) in enumerate(self.segments):
            while self.place[wg] < g:
                yield
            for i in range(u, u + units):
                if wg % team >= self.active[g] and not (self.pl["stream"] and i % 2 != wg // team):
                    yield from self.wait(self.s_full[i % ns], i // ns)
                    yield from self.join(wg, 1)
                    yield from self.free(self.p_empty[i % 2], i // 2)
                    yield from self.join(wg, 1)
                    yield
            u += units

    def softmax(self, wg):
        u = 0
        nv, nc, ns, team = self.pl["NV"], self.pl["NC"], self.pl["NS"], self.pl["team"]
        for g in range(len(self.segments) + 1):
            s = yield from self.take4(g)
            if s is None:
                return
            active = self.active[g]
            self.place[wg] = g
            yield from self.free(self.l_empty[g % 2], g // 2)
            yield from self.wait(self.r_full[g % 2], g // 2)
            for k in range(s[1][0]):
                i, u = u, u + 1
                if self.pl["stream"] and i % 2 != wg // team:
                    continue
                if wg % team >= active and not self.absent:
                    yield from self.wait(self.s_full[i % ns], i // ns)
                    yield from self.join(wg, 0)
                    self.s_empty[i % ns].arrive()
                    self.c_empty[i % nc].arrive()
                    yield from self.free(self.p_empty[i % 2], i // 2)
                    yield from self.join(wg, 0)
                    yield
                    self.p_full[i % 2].arrive()
                    continue
                if wg % team >= active:
                    continue
                yield from self.wait(self.s_full[i % ns], i // ns)
                assert self.buf[("c", i % nc)] == i                 # the scales came with K
                assert self.buf[("s", i % ns)] == i and self.buf[("r", g % 2)] == g
                b, use = i % 2, i // 2
                if not self.pl["stream"]:
                    yield from self.free(self.p_empty[b], use)
                if k >= (2 if self.pl["stream"] else 1) and self.rng.random() < 0.2:          # a reference moves
                    j = i - (2 if self.pl["stream"] else 1)    # the last product into this O^T
                    yield from self.wait(self.p_empty[j % 2], j // 2)
                yield
                for _ in range(1 if not self.absent or wg % team else 1 + team - active):
                    self.s_empty[i % ns].arrive()
                    self.c_empty[i % nc].arrive()
                if self.pl["stream"]:
                    yield from self.free(self.p_empty[b], use)
                if self.buf.setdefault(("p", b), set()) != {i}:
                    self.buf[("p", b)] = {i}
                if k >= s[1][0] - s[1][1] and wg % team == active - 1:
                    yield from self.wait(self.v_full[i % nv], i // nv)
                    assert self.buf[("v", i % nv)] == i
                yield
                for _ in range(1 if not self.absent or wg % team else 1 + team - active):
                    self.p_full[b].arrive()
            self.refs[(g % 2, wg)] = g
            yield
            while self.passed[wg][1] < self.passed[wg][0]:        # the warp joins in any case
                yield
            for _ in range(4):
                self.l_full[g % 2].arrive()

    def split(self, warp, g):
        nq = self.pl["NQ"]
        yield from self.free(self.q_empty[g % nq], g // nq)
        # every softmax warp has left the segment whose rows' powers of two stood there
        assert g < 2 or all(self.refs[(g % 2, w)] >= g - 2 for w in range(self.groups))
        yield
        self.put(("q", g % nq), g)
        self.put(("r", g % 2), g)
        self.q_full[g % nq].arrive()
        self.r_full[g % 2].arrive()

    def results(self, warp):
        g, n = -1, self.pl["SEGS"]
        while True:
            nxt = yield from self.listed(g + 1)
            if nxt is not None:
                yield from self.split(warp, g + 1)
            yield
            if g >= 0:
                assert self.segs[g % n][0] == g                   # still there
                yield from self.wait(self.l_full[g % 2], g // 2)
                assert all(self.refs[(g % 2, w)] == g for w in range(self.groups))
                yield
                yield from self.wait(self.o_full[g % 2], g // 2)
                yield
                assert all(self.refs[(g % 2, w)] == g for w in range(self.groups)) and self.segs[g % n][0] == g
                self.o_empty[g % 2].arrive()
                self.l_empty[g % 2].arrive()
                self.seg_empty[g % n].arrive()
                if warp == 0:
                    self.done_results.append(g)
            if nxt is None:
                return
            g += 1

    def schedule(self, roles):
        live = dict(enumerate(roles))
        slow = self.rng.choice(list(live) + [None, None])        # one role that lags
        lagging = self.rng.choice(["tma", "tmav", "tk", "score", "value"])   # one kind of work that lags
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
            assert idle < 400000, "deadlock"
        while self.pending:
            self.pending.pop(0)[1]()
        assert self.done_results == list(range(len(self.segments)))

    def run(self):
        roles = [self.load_k(), self.load_v(), self.score(), self.value()]
        roles += [self.softmax(w) for w in range(self.groups)] + [self.results(w) for w in range(4)]
        roles += [self.other_lanes(w) for w in range(self.groups)] if not self.absent else []
        self.schedule(roles)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rp", [16, 32, 64])
def test_pipeline_has_no_wrong_phase_no_overwrite_and_no_deadlock(plans, hd, rp):
    pl = plans[hd, rp]
    assert pl["NK"] >= 2 and pl["NV"] >= 2
    for seed in range(60):
        rng = random.Random(seed * 100 + rp + hd)
        # (units, masked units at the end) of each segment
        segments = [(rng.choice([1, 1, 2, 3, 7, 20]), rng.choice([0, 1, 2])) for _ in range(rng.choice([1, 2, 6, 12]))]
        Model8(pl, segments, rng).run()


def test_the_model_rejects_powers_of_two_without_their_own_barrier(plans):
    """The softmax waiting for the query tile's barrier with one tile instead of two: it
    is refilled before every softmax warp has looked, and the parity reads as another
    phase's.  The model has to see it."""
    class Shared(Model8):
        def wait(self, bar, k):
            for par in (0, 1):
                if bar is self.r_full[par]:
                    return super().wait(self.q_full[0], 2 * k + par)
            return super().wait(bar, k)

    wrong = 0
    for seed in range(40):
        try:
            Shared(dict(plans[128, 64], NQ=1), [(1, 0)] * 8, random.Random(seed)).run()
        except AssertionError:
            wrong += 1
    assert wrong > 0


def test_the_model_rejects_warpgroups_that_miss_phases(plans):
    """Warpgroups without rows that sit a segment out come back with the parity of a phase
    that lies ahead."""
    class Absent(Model8):
        absent = True

    wrong = 0
    for seed in range(40):
        try:
            Absent(plans[64, 64], [(7, 0)] * 8, random.Random(seed)).run()
        except AssertionError:
            wrong += 1
    assert wrong > 0


def test_the_model_rejects_a_warp_whose_lanes_do_not_join(plans):
    """The lane that arrives for the warp lets the next phase end before the others have
    looked at this one."""
    class Apart(Model8):
        apart = True

    wrong = 0
    for seed in range(40):
        try:
            Apart(plans[64, 64], [(7, 0)] * 8, random.Random(seed)).run()
        except AssertionError:
            wrong += 1
    assert wrong > 0
