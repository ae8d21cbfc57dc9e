"""The 8-bit attention's pipeline on the host: its shared-memory plan, compiled from
the kernel's own header, and its roles as coroutines under random schedules, as
test_paged_pipeline_cpu.py runs the bf16 kernel's.

What is new against that model: the results' warps split the next segment's queries
before they write a segment's results (q_full, and r_full for what the softmax needs
of the rows), scales have a ring of their own, and a warpgroup frees its chunk's
scales with its S^T."""
import os
import random
import subprocess

import pytest

from test_paged_pipeline_cpu import SEGS, Barrier, Model

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = r"""
#include <stdio.h>
#include "paged_plan8.h"
using namespace sv::plan8;
template <int HD, int RP> void line() {
    using L = Plan<HD, RP>;
    printf("%d %d %d %d %d %d %d %d %d %d %d\n", HD, RP, (int)sizeof(Fixed<RP>), L::kBytes, L::NK, L::NV, L::NQ, L::NP, kScaleSlots, (int)L::kStream, L::kUsed);
}
int main() {
    line<64, 16>(); line<64, 32>(); line<64, 64>(); line<64, 128>();
    line<128, 16>(); line<128, 32>(); line<128, 64>(); line<128, 128>();
}
"""
NAMES = ["HD", "RP", "fixed", "bytes", "NK", "NV", "NQ", "NP", "NC", "stream", "columns"]


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan8")
    (d / "plan.cpp").write_text(SRC)
    inc = os.path.join(ROOT, "speculative_decoding_verify_pass_gb300", "csrc")
    subprocess.check_call(["g++", "-std=c++17", "-I", inc, str(d / "plan.cpp"), "-o", str(d / "plan")])
    rows = [dict(zip(NAMES, map(int, x.split()))) for x in subprocess.check_output([str(d / "plan")]).decode().split("\n") if x]
    return {(r["HD"], r["RP"]): dict(r, pieces=1) for r in rows}


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rp", [16, 32, 64, 128])
def test_static_memory_and_tiles_fit(plans, hd, rp):
    r = plans[hd, rp]
    assert r["fixed"] + r["bytes"] <= 227 * 1024 and r["columns"] <= 512
    # K, V, both parts of the queries, three parts of P^T, up to 1 KB of alignment and 1 KB behind the last V
    chunk = 128 * hd
    assert r["bytes"] >= (r["NK"] + r["NV"]) * chunk + r["NQ"] * 2 * rp * hd + r["NP"] * 3 * 128 * rp + 2048
    groups = 2 if r["stream"] else 1
    # scales of 8 chunks; per row: references and four sums of two parities and up to two groups, powers of two, weights, token, offset
    assert r["fixed"] >= 8 * 256 + rp * (2 * groups * 5 * 4 + 2 * 4 + 2 * 8 + 4 + 8) + 4 * 1025
    # a slot of scales is always read by the same warpgroup (it then sees every phase of its barrier)
    assert r["NC"] % 2 == 0


class Model8(Model):
    def __init__(self, pl, segments, rng):
        super().__init__(pl, segments, rng)
        n = lambda k, c=1: [Barrier(c) for _ in range(k)]  # noqa: E731
        self.q_full, self.r_full = n(pl["NQ"], 4), n(2, 4)
        self.c_full, self.c_empty = n(pl["NC"]), n(pl["NC"], 4 if pl["stream"] else 8)

    def load_k(self):
        u, nk, nc = 0, self.pl["NK"], self.pl["NC"]
        for g in range(len(self.segments) + 1):
            yield from self.free(self.seg_empty[g % SEGS], g // SEGS)
            self.segs[g % SEGS] = (g, self.segments[g]) if g < len(self.segments) else None
            self.seg_full[g % SEGS].arrive()
            if g == len(self.segments):
                return
            for _ in range(self.segments[g][0]):
                yield from self.free(self.c_empty[u % nc], u // nc)
                yield from self.free(self.k_empty[u % nk], u // nk)
                self.async_("tk", lambda u=u: (self.put(("c", u % nc), u), self.c_full[u % nc].arrive()))
                self.async_("tma", lambda u=u: (self.put(("k", u % nk), u), self.k_full[u % nk].arrive()))
                u += 1
                yield

    def softmax(self, warp):
        wg, u = warp // 4, 0
        nv, nc, np_ = self.pl["NV"], self.pl["NC"], self.pl["NP"]
        for g in range(len(self.segments) + 1):
            s = yield from self.take(g)
            if s is None:
                return
            yield from self.free(self.l_empty[g % 2], g // 2)
            yield from self.wait(self.r_full[g % 2], g // 2)
            for k in range(s[1][0]):
                i, u = u, u + 1
                if self.pl["stream"] and i % 2 != wg:
                    continue
                yield from self.wait(self.c_full[i % nc], i // nc)
                assert self.buf[("c", i % nc)] == i
                yield from self.wait(self.s_full[i % 2], i // 2)
                assert self.buf[("s", i % 2)] == i and self.buf[("r", g % 2)] == g
                b, use = (i % 2, i // 2) if self.pl["stream"] else (0, i)
                if k > 1 and self.rng.random() < 0.2:          # a reference moves
                    yield from self.free(self.p_empty[b], use)
                yield
                self.s_empty[i % 2].arrive()
                self.c_empty[i % nc].arrive()
                yield from self.free(self.p_empty[b], use)
                if self.buf.setdefault(("p", b), set()) != {i}:
                    self.buf[("p", b)] = {i}
                if k >= s[1][0] - s[1][1] and (self.pl["stream"] or wg == 0):
                    yield from self.wait(self.v_full[i % nv], i // nv)
                    assert self.buf[("v", i % nv)] == i
                yield
                self.p_full[b].arrive()
            self.refs[(g % 2, warp)] = g
            yield
            self.l_full[g % 2].arrive()

    def split(self, warp, g):
        nq = self.pl["NQ"]
        yield from self.free(self.q_empty[g % nq], g // nq)
        # every softmax warp has left the segment whose rows' powers of two stood there
        assert g < 2 or all(self.refs[(g % 2, w)] >= g - 2 for w in range(8))
        yield
        self.put(("q", g % nq), g)
        self.put(("r", g % 2), g)
        self.q_full[g % nq].arrive()
        self.r_full[g % 2].arrive()

    def results(self, warp):
        s = yield from self.take(0)
        if s is not None:
            yield from self.split(warp, 0)
        g = 0
        while s is not None:
            s = yield from self.take(g + 1)
            if s is not None:
                yield from self.split(warp, g + 1)
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
            g += 1


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rp", [16, 32, 64, 128])
def test_pipeline_has_no_wrong_phase_no_overwrite_and_no_deadlock(plans, hd, rp):
    pl = plans[hd, rp]
    assert pl["NK"] >= 2 and pl["NV"] >= 2
    for seed in range(60):
        rng = random.Random(seed * 100 + rp + hd)
        # (units, masked units at the end) of each segment
        segments = [(rng.choice([1, 1, 2, 3, 7, 20]), rng.choice([0, 1, 2])) for _ in range(rng.choice([1, 2, 6, 12]))]
        Model8(pl, segments, rng).run()


def test_the_model_rejects_powers_of_two_without_their_own_barrier(plans):
    """The softmax waiting for the query tile's barrier instead: a tile of short segments
    is refilled before every softmax warp has looked, and the parity reads as another
    phase's.  The model has to see it."""
    class Shared(Model8):
        def wait(self, bar, k):
            for par in (0, 1):
                if bar is self.r_full[par]:
                    g = 2 * k + par
                    return super().wait(self.q_full[g % self.pl["NQ"]], g // self.pl["NQ"])
            return super().wait(bar, k)

    pl = dict(plans[128, 128])
    assert pl["NQ"] == 1
    wrong = 0
    for seed in range(40):
        try:
            Shared(pl, [(1, 0)] * 8, random.Random(seed)).run()
        except AssertionError:
            wrong += 1
    assert wrong > 0
