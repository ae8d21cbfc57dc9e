"""The 8-bit attention's split of work over CTAs, compiled for the host from the
kernel's own header: every chunk of every pair is in exactly one segment, the units
in front of a pair belong to no segment, each split pair's partials are the ones its
owner joins, and blocks cover a sequence's rows."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = r"""
#include "paged_split8.h"
using namespace sv::split8;
extern "C" {
int head() { return kHead; }
int chunks(int len) { return chunks_of(len); }
int blocks(int rows, int group, int tile) { return blocks_of(rows, group, tile_tokens(tile, group)); }
long long units(int rows, int len, int group, int tile, int hkv) { return units_of(rows, len, group, tile_tokens(tile, group), hkv); }
int begin(int c, int total, int ctas) { return Deal(total, ctas).begin(c); }
int c0(int u0, int u1) { return part_of(u0, u1).c0; }
int c1(int u0, int u1) { return part_of(u0, u1).c1; }
int owner(int total, int ctas, int begin) { return owner_of(Deal(total, ctas), begin); }
int parts(int total, int ctas, int begin, int chunks) { Deal d(total, ctas); return parts_of(d, owner_of(d, begin), begin, chunks); }
void place(int block, int group, int tile, int* out) { Place p; p.at(block, group, tile_tokens(tile, group)); out[0] = p.token; out[1] = p.skip; }
void step(int group, int tile, int* out) { Place p = {out[0], out[1]}; p.step(group, tile_tokens(tile, group)); out[0] = p.token; out[1] = p.skip; }
int height(int group, int max_new) { return tile_height(group, max_new); }
int tile(int height, int group) { return tile_rows(height, group); }
}
"""


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    d = tmp_path_factory.mktemp("split8")
    (d / "split.cpp").write_text(SRC)
    inc = os.path.join(ROOT, "speculative_decoding_verify_pass_gb300", "csrc")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", inc, str(d / "split.cpp"), "-o", str(d / "split.so")])
    lib = ctypes.CDLL(str(d / "split.so"))
    lib.units.restype = ctypes.c_longlong
    return lib


CASES = [([300], [1], 8, 4, 1, 152), ([4104], [8], 8, 4, 8, 152), ([1], [1], 1, 1, 1, 152), ([0, 0], [1, 0], 2, 4, 1, 152), ([100003], [1], 8, 4, 1, 152),
         ([128 * 152], [1], 1, 16, 1, 152), ([7, 0, 900, 128, 129], [0, 3, 40, 16, 2], 3, 4, 16, 152), ([5, 6], [0, 0], 4, 4, 1, 152),
         ([400], [130], 4, 1, 16, 152), ([256] * 7, [1] * 7, 11, 2, 1, 5), ([3000, 50], [3, 2], 1, 128, 3, 152), ([700] * 9, [5] * 9, 2, 100, 1, 40)]


def random_case(rng):
    n = rng.choice([1, 2, 30, 400, 1024])
    return ([rng.choice([0, 1, 127, 128, 129, rng.randint(0, 5000)]) for _ in range(n)], [rng.randint(0, 20) for _ in range(n)],
            rng.choice([1, 2, 8]), rng.choice([1, 2, 3, 4, 16, 65, 128]), rng.choice([1, 8, 16]), rng.choice([1, 4, 152]))


ALL = CASES + [random_case(random.Random(i)) for i in range(16)]


@pytest.mark.parametrize("case", ALL, ids=lambda c: "%dx%dx%d" % (len(c[0]), c[2], c[3]))
def test_segments_partition_the_chunks_and_partials_meet_their_owner(split, case):
    lens, rows, hkv, group, hint, ctas = case
    tile = split.tile(split.height(group, hint), group)
    E = split.head()
    pairs, at = [], 0                                 # (first unit, chunks)
    for n, m in zip(lens, rows):
        c, b = max(1, -(-n // 128)), -(-m * group // tile)
        assert split.chunks(n) == c and split.blocks(m, group, tile) == b
        assert split.units(m, n, group, tile, hkv) == b * hkv * (c + E)
        for _ in range(b * hkv):
            pairs.append((at, c))
            at += c + E
    T = at
    got = {}                                          # pair -> [(cta, chunks, slot)]
    taken_whole = []
    i = 0
    for c in range(ctas):
        a, b = split.begin(c, T, ctas), split.begin(c + 1, T, ctas)
        u, first, parts = a, True, []
        while i and pairs and i < len(pairs) and pairs[i][0] > a:
            i -= 1
        while i + 1 < len(pairs) and pairs[i][0] + pairs[i][1] + E <= a:
            i += 1
        while u < b:
            p0, n = pairs[i]
            u0, u1 = u - p0, min(n + E, b - p0)
            c0, c1 = split.c0(u0, u1), split.c1(u0, u1)
            assert 0 <= c0 <= c1 <= n
            if u0 == 0:
                taken_whole.append(i)
            if c1 > c0:
                slot = -1 if (c0, c1) == (0, n) else 2 * c + (0 if c0 > 0 else 1)
                got.setdefault(i, []).append((c, c0, c1, slot))
                parts.append((i, c0, c1))
            u = p0 + u1
            if u == p0 + n + E:
                i += 1
        # at most one pair that goes on into a CTA (its first), one that begins in it and goes on (its last)
        for k, (j, c0, c1) in enumerate(parts):
            assert c0 == 0 or k == 0
            assert c1 == pairs[j][1] or k == len(parts) - 1
    assert taken_whole == list(range(len(pairs)))     # whole pairs: each by the CTA it begins in
    slots = set()
    for j, (p0, n) in enumerate(pairs):
        segs = got[j]
        assert [x for _, c0, c1, _ in segs for x in range(c0, c1)] == list(range(n))
        if len(segs) == 1:
            assert segs[0][3] == -1
            continue
        owner = split.owner(T, ctas, p0)
        assert owner == segs[0][0] and split.parts(T, ctas, p0, n) == len(segs)
        for t, (c, _, _, slot) in enumerate(segs):
            assert c == owner + t and slot == (2 * owner + 1 if t == 0 else 2 * (owner + t))
            assert slot not in slots
            slots.add(slot)


@pytest.mark.parametrize("group", [1, 2, 3, 4, 7, 8, 16, 40, 63, 64, 65, 100, 127, 128])
def test_tiles_and_blocks_cover_the_rows(split, group):
    for hint in (1, 2, 3, 8, 16, 17, 1000, 2 ** 31 - 1):
        h = split.height(group, hint)
        assert h in (16, 32, 64) and (h == 16 or h // 2 < group * hint) and h >= min(64, group * hint)
        tile = split.tile(h, group)
        assert 1 <= tile <= h and (tile % group == 0 or group > 64 and tile == 64)
        for rows in (1, 2, 5, 33):
            seen = []
            for b in range(split.blocks(rows, group, tile)):
                r0 = b * tile
                skip = r0 - r0 // group * group
                n = min(tile, rows * group - r0)
                assert n > 0 and (group > h or skip == 0)
                for r in range(n):
                    t = (skip + r) // group           # token counted from the block's first
                    assert t == (int(skip + r >= group) if group > h else r // group)
                    seen.append((r0 // group + t, skip + r - t * group))
            assert seen == [(t, g) for t in range(rows) for g in range(group)]


@pytest.mark.parametrize("group", [1, 3, 4, 16, 33, 63, 64, 65, 100, 127, 128])
@pytest.mark.parametrize("hint", [1, 4, 1000])
def test_blocks_begin_where_the_flattened_rows_say(split, group, hint):
    tile = split.tile(split.height(group, hint), group)
    at, walked = (ctypes.c_int * 2)(), (ctypes.c_int * 2)(0, 0)
    for block in range(500):
        split.place(block, group, tile, at)
        assert tuple(at) == divmod(block * tile, group) == tuple(walked)
        split.step(group, tile, walked)
    for block in (10 ** 6, 2 ** 24 - 1, 2 ** 31 // max(1, tile // group) - 1):
        split.place(block, group, tile, at)
        assert tuple(at) == divmod(block * tile, group)
