"""Paged attention's shared memory, compiled for the host from the kernels' own
header: what a CTA keeps in static memory and the tiles beside it fit for every
instance, by the declarations themselves, and the buffer counts are those that
the pipeline's model runs with."""
import os
import subprocess

import pytest

from test_paged_pipeline_cpu import plan

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = r"""
#include <stdio.h>
#include <stdlib.h>
#include "paged_plan.h"
using namespace sv::plan;
template <int HD, int RP> void line() {
    using L = Plan<HD, RP>;
    printf("%d %d %d %d %d %d %d %d %d %d\n", HD, RP, (int)sizeof(Fixed<RP>), L::kBytes, L::NK, L::NV, L::NQ, L::NP, L::kPieces, (int)L::kStream);
}
int main(int argc, char** argv) {
    for (int i = 1; i < argc; ++i) printf("%d\n", wait_rounds(atoi(argv[i])));
    if (argc > 1) return 0;
    line<64, 16>(); line<64, 32>(); line<64, 64>(); line<64, 128>();
    line<128, 16>(); line<128, 32>(); line<128, 64>(); line<128, 128>();
}
"""
NAMES = ["HD", "RP", "fixed", "bytes", "NK", "NV", "NQ", "NP", "pieces", "stream"]


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SRC)
    inc = os.path.join(ROOT, "speculative_decoding_verify_pass_gb300", "csrc")
    subprocess.check_call(["g++", "-std=c++17", "-I", inc, str(d / "plan.cpp"), "-o", str(d / "plan")])
    return str(d / "plan")


@pytest.fixture(scope="module")
def plans(program):
    out = subprocess.check_output([program]).decode().split("\n")
    rows = [dict(zip(NAMES, map(int, x.split()))) for x in out if x]
    return {(r["HD"], r["RP"]): r for r in rows}


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rp", [16, 32, 64, 128])
def test_static_memory_and_tiles_fit(plans, hd, rp):
    r = plans[hd, rp]
    assert r["fixed"] + r["bytes"] <= 227 * 1024
    # the tiles: K, V, queries, both parts of P^T, up to 1 KB of alignment and 1 KB behind the last V
    chunk = 128 * hd * 2
    assert r["bytes"] >= r["NK"] * chunk + r["NV"] * chunk // r["pieces"] + r["NQ"] * rp * hd * 2 + r["NP"] * 2 * 128 * rp * 2 + 2048
    # per row: reference and four sums of two segment parities and up to two groups, weights, token, offset
    groups = 2 if r["stream"] else 1
    assert r["fixed"] >= rp * (2 * groups * 5 * 4 + 2 * 8 + 4 + 8) + 4 * 1025


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rp", [16, 32, 64, 128])
def test_buffer_counts_are_the_model_s(plans, hd, rp):
    r, model = plans[hd, rp], plan(hd, rp)
    assert {k: r[k] for k in ("NK", "NV", "NQ", "NP", "pieces")} == {k: model[k] for k in ("NK", "NV", "NQ", "NP", "pieces")}
    assert bool(r["stream"]) == model["stream"]


def test_results_are_waited_for_as_long_as_their_chunks_take(program):
    """The longest table's sequence is 2^19 chunks, and one CTA's segment may hold them all: at
    17000 cycles a chunk (each takes its scores again) that is four times one wait's 2^31.  Every
    chunk gets 2^16 cycles at least."""
    units = [1, 2, 1000, 32767, 32768, 65535, 65536, 300001, 2 ** 19]
    rounds = list(map(int, subprocess.check_output([program] + list(map(str, units))).split()))
    assert 2 ** 19 * 17000 > 4 * 2 ** 31
    assert all(r * 2 ** 31 >= u * 2 ** 16 for u, r in zip(units, rounds))
    assert rounds[0] == 1 and max(rounds) <= 17           # a second as a rule, some seconds at most
