"""The three e5m2 parts that the 8-bit attention makes of a weight (a half), restated for
every half: what they leave, and that none of them overflows."""
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BORDER = 0x7B80        # halves from here on (61440) round to e5m2's infinity: their chunk is taken again


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("weights8")
    (d / "w.cpp").write_text('#include <stdio.h>\n#include "paged_plan8.h"\nusing namespace sv::plan8;\n'
                             'int main() { printf("%d %d %d", kShift8, kPart2, kPart3); }\n')
    inc = os.path.join(ROOT, "speculative_decoding_verify_pass_gb300", "csrc")
    subprocess.check_call(["g++", "-std=c++17", "-I", inc, str(d / "w.cpp"), "-o", str(d / "w")])
    return [int(x) for x in subprocess.check_output([str(d / "w")]).split()]


def upper(bits):
    """The e5m2 number in a half's upper byte."""
    return (bits & 0xFF00).astype(np.uint16).view(np.float16)


def parts(bits, m2, m3):
    h = bits.view(np.float16)
    p1 = upper(bits + 0x80)
    r = (h - p1) * np.float16(m2)
    p2 = upper(r.view(np.uint16) + 0x80)
    r = (r - p2) * np.float16(m3)
    return p1, p2, upper(r.view(np.uint16) + 0x80)


def test_parts_of_every_half(plan):
    _, m2, m3 = plan
    bits = np.arange(BORDER, dtype=np.uint16)
    p1, p2, p3 = (p.astype(np.float64) for p in parts(bits, m2, m3))
    assert all(np.isfinite(p).all() and np.abs(p).max() <= 57344 for p in (p1, p2, p3))
    h = bits.view(np.float16).astype(np.float64)
    left = np.abs(p1 + (p2 + p3 / m3) / m2 - h)
    power = np.exp2(np.floor(np.log2(np.maximum(h, 2.0 ** -24))))
    # half of a third part's last bit, 2^-3 of at most the weight's power over m2 m3; where e5m2 ends half of its smallest step
    assert (left <= np.maximum(2.0 ** -11 * power, 2.0 ** -17 / (m2 * m3))).all()
    assert 2.0 ** -17 / (m2 * m3) <= 2.0 ** -24


def test_halves_at_the_border():
    """The next half's first part would be infinite; the vote's test sees exactly those, and NaN."""
    bits = np.array([BORDER - 1, BORDER, 0x7BFF, 0x7C00, 0x7FFF], dtype=np.uint16)
    assert np.isfinite(upper(bits[:1] + 0x80)).all() and np.isinf(upper(bits[1:2] + 0x80)).all()
    assert ((bits + 0x0480) & 0x8000 != 0).tolist() == [False, True, True, True, True]
