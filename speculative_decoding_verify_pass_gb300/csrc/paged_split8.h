// How the 8-bit paged attention's work is dealt to CTAs (host and device; the host
// side is what the tests drive).
//
// As in paged_split.h a unit is one 128-position chunk of one pair (row block, kv
// head), and C CTAs work on equal ranges of the units in order.  Two things differ.
//
// A row block is up to `tile` rows of the flattened (token, query head of the kv
// head) order: whole tokens while a token's heads fit a tile, else parts of one or
// two tokens (the block's first row is then head `skip` of its first token).
//
// A pair begins with kHead units that are no chunk: a segment costs about as much
// beside its chunks (queries, references, sums, results), and CTAs with many short
// segments would end late (64 ragged decodes: 104 us with one such unit, 95 with four;
// 24 sequences of 16 new rows: 206 and 154).  A CTA whose range holds only such units of a pair does
// not work on it; the CTA that holds its first chunk owns it.
#pragma once

#include "paged_split.h"

namespace sv {
namespace split8 {

using split::chunks_of;
using split::Deal;
using split::kChunk;

constexpr int kHead = 4;                // units in front of a pair's chunks
constexpr int kMostRows = 64;           // of a tile

// Tile height that the kernel is compiled for, and the rows of a block in it.
SPLIT_HD int tile_height(int group, int max_new) {
    const int64_t want = (int64_t)group * max_new;
    return want <= 16 ? 16 : want <= 32 ? 32 : kMostRows;
}
SPLIT_HD int tile_rows(int height, int group) { return group <= height ? height / group * group : height; }

SPLIT_HD int blocks_of(int rows, int group, int tile) { return (int)(((int64_t)rows * group + tile - 1) / tile); }
SPLIT_HD int64_t units_of(int rows, int len, int group, int tile, int hkv) {
    return (int64_t)blocks_of(rows, group, tile) * hkv * (chunks_of(len) + kHead);
}

// The part of a pair that units [u0, u1) of it (counted from its first one) cover.
struct Part {
    int c0, c1;                         // chunks
};
SPLIT_HD Part part_of(int u0, int u1) {
    Part p;
    p.c0 = u0 > kHead ? u0 - kHead : 0;
    p.c1 = u1 > kHead ? u1 - kHead : 0;
    return p;
}
// The CTA that holds the first chunk of a pair whose first unit is `begin`, and how
// many CTAs work on it.
SPLIT_HD int owner_of(const Deal& d, int begin) { return d.cta(begin + kHead); }
SPLIT_HD int parts_of(const Deal& d, int begin, int chunks) { return d.parts(owner_of(d, begin), begin + kHead + chunks); }

}  // namespace split8
}  // namespace sv
