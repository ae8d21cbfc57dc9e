"""Paged attention's split of work over CTAs, compiled for the host from the
kernels' own header: every unit of every pair is in exactly one segment, each
split pair's partials are the ones its owner joins, and no two segments share a
slot."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = r"""
#include "paged_split.h"
using namespace sv::split;
extern "C" {
int chunks(int len) { return chunks_of(len); }
int blocks(int rows, int tokens) { return blocks_of(rows, tokens); }
long long units(int rows, int len, int tokens, int hkv) { return units_of(rows, len, tokens, hkv); }
int work(int ctas, int total) { return Deal(total, ctas).work; }
int begin(int c, int total, int ctas) { return Deal(total, ctas).begin(c); }
int cta(int u, int total, int ctas) { return Deal(total, ctas).cta(u); }
int sequence(const int* first, int nseq, int u) { return sequence_of(first, nseq, u); }
int parts(int c, int pair_end, int total, int ctas) { return Deal(total, ctas).parts(c, pair_end); }
int tile(int group, int max_new) { return tile_rows(group, max_new); }
}
"""


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    d = tmp_path_factory.mktemp("split")
    (d / "split.cpp").write_text(SRC)
    inc = os.path.join(ROOT, "speculative_decoding_verify_pass_gb300", "csrc")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", inc, str(d / "split.cpp"), "-o", str(d / "split.so")])
    lib = ctypes.CDLL(str(d / "split.so"))
    lib.units.restype = ctypes.c_longlong
    return lib


CASES = [([300], [1], 8, 16, 152), ([4104], [8], 8, 4, 152), ([1], [1], 1, 16, 152), ([0, 0], [1, 0], 2, 4, 152), ([100003], [1], 8, 4, 152),
         ([128 * 152], [1], 1, 16, 152), ([128 * 151 + 1], [1], 1, 16, 152), ([7, 0, 900, 128, 129], [0, 3, 40, 16, 2], 3, 4, 152),
         ([5, 6], [0, 0], 4, 4, 152), ([400], [130], 4, 1, 152), ([256] * 7, [1] * 7, 11, 2, 5)]


def random_case(rng):
    n = rng.choice([1, 2, 30, 400, 1024])
    return ([rng.choice([0, 1, 127, 128, 129, rng.randint(0, 5000)]) for _ in range(n)], [rng.randint(0, 20) for _ in range(n)],
            rng.choice([1, 2, 8]), rng.choice([1, 2, 4, 16]), rng.choice([1, 4, 152]))


@pytest.mark.parametrize("case", CASES + [random_case(random.Random(i)) for i in range(12)], ids=lambda c: "%dx%d" % (len(c[0]), c[2]))
def test_segments_partition_the_units_and_partials_meet_their_owner(split, case):
    lens, rows, hkv, tokens, ctas = case
    first = [0]
    pairs = []                                        # (first unit, last unit + 1)
    for n, m in zip(lens, rows):
        c, b = split.chunks(n), split.blocks(m, tokens)
        assert c == max(1, -(-n // 128)) and b == -(-m // tokens)
        assert split.units(m, n, tokens, hkv) == b * hkv * c
        pairs += [(first[-1] + k * c, first[-1] + (k + 1) * c) for k in range(b * hkv)]
        first.append(first[-1] + b * hkv * c)
    T = first[-1]
    arr = (ctypes.c_int * len(first))(*first)
    w = split.work(ctas, T)
    assert w == min(ctas, T)
    written = {}                                      # slot -> (pair, units)
    whole = set()
    at = 0
    pair_of = {}
    for i, (a, b) in enumerate(pairs):
        for u in range(a, b):
            pair_of[u] = i
    metas = []
    for c in range(ctas):
        a, b = split.begin(c, T, ctas), split.begin(c + 1, T, ctas)
        assert a == at and (b - a in (T // w, T // w + 1) if c < w else b == a)
        at = b
        u = a
        last = None
        while u < b:
            q = split.sequence(arr, len(lens), u)
            assert first[q] <= u < first[q + 1]
            i = pair_of[u]
            assert split.cta(u, T, ctas) == c and split.cta(pairs[i][0], T, ctas) <= c
            e = min(b, pairs[i][1])
            if (u, e) == pairs[i]:
                whole.add(i)
            else:
                slot = 2 * c + (0 if u == a else 1)
                assert slot not in written
                written[slot] = (i, range(u, e))
            last = (i, u, e)
            u = e
        if last and last[2] < pairs[last[0]][1] and pairs[last[0]][0] >= a:
            i = last[0]
            metas.append((i, c, 2 * c + (0 if pairs[i][0] == a else 1), split.parts(c, pairs[i][1], T, ctas)))
    assert at == T
    joined = set()
    for i, c, slot, count in metas:
        got = []
        for t in range(count):
            s = slot if t == 0 else 2 * (c + t)
            assert written[s][0] == i
            got += list(written[s][1])
            joined.add(s)
        assert got == list(range(*pairs[i]))
    assert joined == set(written)
    assert len(whole) + len(metas) == len(pairs)


@pytest.mark.parametrize("case", CASES + [random_case(random.Random(i)) for i in range(12)], ids=lambda c: "%dx%d" % (len(c[0]), c[2]))
def test_whole_pairs_are_each_taken_by_the_cta_they_begin_in(split, case):
    lens, rows, hkv, tokens, ctas = case
    starts, at = [], 0
    for n, m in zip(lens, rows):
        for _ in range(split.blocks(m, tokens) * hkv):
            starts.append(at)
            at += split.chunks(n)
    taken = []
    for c in range(ctas):
        a, b = split.begin(c, at, ctas), split.begin(c + 1, at, ctas)
        taken += [u for u in starts if a <= u < b]
    assert taken == starts


def test_tile_rows(split):
    for g in range(1, 129):
        for n in (1, 2, 3, 8, 16, 17, 1000, 2 ** 31 - 1):
            t = split.tile(g, n)
            assert t in (16, 32, 64, 128) and t // g >= 1
            assert t >= min(128, g * n) and (t == 16 or t // 2 < g * n)
