"""Waits of the 8-bit attention that last a segment, on the host: the roles of
test_paged8_giveup_cpu.py with segments that take several limits of a wait.  The results'
warps, and softmax warps that have no rows and do not keep up with the barriers, wait for
the next entry of the list from the start of a segment to its last copy of K."""
import os
import random
import re
import subprocess

import pytest

from test_paged8_giveup_cpu import Cta8
from test_paged8_pipeline_cpu import plans  # noqa: F401  (a fixture)

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_verify_pass_gb300", "csrc")


class Long(Cta8):
    """Waits for the list are given `listed` limits (a function of the units of the segment before), of
    the results' warps (`late` False: theirs alone) and of all others; every other wait has one."""
    late = True

    def __init__(self, pl, segments, rng, lost, listed):
        super().__init__(pl, segments, rng, lost)
        self.listed = listed

    def take(self, g):
        rounds = self.listed(self.segments[g - 1][0] if g and self.late else 0)
        yield from self.wait(self.seg_full[g % self.S], (g // self.S) % 2, rounds)
        s = self.segs[g % self.S]
        yield
        self.seg_empty[g % self.S].arrive()
        return s

    def results(self, warp):
        g, group = -1, self.groups[-1]
        while True:
            rounds = self.listed(self.segments[g][0] if g >= 0 else 0)
            yield from self.wait(self.seg_full[(g + 1) % self.S], ((g + 1) // self.S) % 2, rounds)
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
                    yield from self.wait(self.l_full[g % 2], (g // 2) % 2, 1 + self.segments[g][0] // 8)
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


SHAPES = [(64, 16), (128, 32), (128, 64)]


def run(plans, hd, rp, listed, cls=Long):  # noqa: F811
    out = []
    for seed in range(3):
        rng = random.Random(seed)
        segments = [(rng.choice([1, 3, 150, 260]), rng.choice([0, 2])) for _ in range(3)] + [(200, 1)]
        rng.shuffle(segments)
        cta = cls(plans[hd, rp], segments, rng, None, listed)
        out.append((cta.run(), cta.time))
    return out


@pytest.mark.parametrize("hd,rp", SHAPES)
def test_long_segments_are_waited_for(plans, hd, rp):  # noqa: F811
    got = run(plans, hd, rp, lambda units: 1 + units // 8)
    assert not any(dead for dead, _ in got)
    assert max(time for _, time in got) > 2 * 4000       # (a segment takes longer than one limit)


def test_the_model_rejects_one_limit_for_the_list(plans):  # noqa: F811
    class Late(Long):
        late = False

    assert any(dead for dead, _ in run(plans, 128, 64, lambda units: 1))
    assert any(dead for dead, _ in run(plans, 64, 16, lambda units: 1))
    assert any(dead for dead, _ in run(plans, 128, 64, lambda units: 1 + units // 8, Late))


def test_limits_of_a_segment(tmp_path):
    """2^16 cycles for each chunk, however many there are; and the kernel gives them to each of these waits."""
    (tmp_path / "r.cpp").write_text('#include <stdio.h>\n#include "paged_plan8.h"\nint main() { for (int u = 0; u <= 1 << 19; u += 1 << 12) '
                                    'printf("%d %d\\n", u, sv::plan8::wait_rounds(u)); }\n')
    subprocess.check_call(["g++", "-std=c++17", "-I", CSRC, str(tmp_path / "r.cpp"), "-o", str(tmp_path / "r")])
    for line in subprocess.check_output([str(tmp_path / "r")]).decode().split("\n")[:-1]:
        units, rounds = map(int, line.split())
        assert rounds >= 1 and rounds * 2 ** 31 >= units * 2 ** 16
    with open(os.path.join(CSRC, "paged_attn8.cu")) as f:
        waits = re.findall(r"wait\(BAR\((?:seg_full|l_full),[^;]*;", f.read())
    assert len(waits) == 3 and all("wait_rounds(" in w for w in waits)
