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
// segments would end late (64 ragged decodes: 104 us with one such unit, 95 with four then;
// 24 sequences of 16 new rows: 206 and 154).  A CTA whose range holds only such units of a pair does
// not work on it; the CTA that holds its first chunk owns it.
//
// Pairs of short tables are left whole by the bf16 calls' rule (split::whole_pairs, up to
// 1024 positions), which holds here too: 8 kv heads of 128, decode, every sequence
// full, split against whole in us with 1, 16 and 64 sequences: 512 positions 7.7 / 6.7,
// 11.7 / 8.5, 22.6 / 18.3; 1024 8.5 / 8.1, 13.8 / 10.2, 31.2 / 29.1; 2048 9.2 / 11.2,
// 15.6 / 13.2, 50.2 / 49.7; 4096 9.6 / 17.3, 29.6 / 26.0, 89.5 / 90.0.
#pragma once

#include "paged_split.h"

namespace sv {
namespace split8 {

using split::chunks_of;
using split::Deal;
using split::kChunk;

constexpr int kHead = 4;                // units in front of a pair's chunks
constexpr int kMostRows = 64;           // of a tile: 128 rows' S^T, O^T and their parts do not fit tensor memory

// Tile height that the kernel is compiled for, and the rows of a block in it.
SPLIT_HD int tile_height(int group, int max_new) {
    const int64_t want = (int64_t)group * max_new;
    return want <= 16 ? 16 : want <= 32 ? 32 : kMostRows;
}
SPLIT_HD int tile_rows(int height, int group) { return group <= height ? height / group * group : height; }

// Whole tokens of a block; 0: a token's heads fill more than one (kMostRows at a time).
SPLIT_HD int tile_tokens(int tile, int group) { return group <= tile ? tile / group : 0; }

SPLIT_HD int blocks_of(int rows, int group, int tokens) {
    if (tokens) return rows > 0 ? (int)((unsigned)(rows - 1) / (unsigned)tokens) + 1 : 0;
    return (int)(((int64_t)rows * group + kMostRows - 1) / kMostRows);
}
SPLIT_HD int64_t units_of(int rows, int len, int group, int tokens, int hkv) {
    return (int64_t)blocks_of(rows, group, tokens) * hkv * (chunks_of(len) + kHead);
}

// Where a block begins: a token, and a query head of it.
struct Place {
    int token, skip;
    SPLIT_HD void at(int block, int group, int tokens) {
        if (tokens) {
            token = block * tokens;
            skip = 0;
        } else {                        // block * kMostRows / group, in 32 bits
            const int whole = block / group, rest = (block - whole * group) * kMostRows;
            token = whole * kMostRows + rest / group;
            skip = rest % group;
        }
    }
    SPLIT_HD void step(int group, int tokens) {     // to the next block
        token += tokens;
        if (!tokens && (skip += kMostRows) >= group) skip -= group, ++token;
    }
};

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
SPLIT_HD int parts_of(const Deal& d, int owner, int begin, int chunks) { return d.parts(owner, begin + kHead + chunks); }

}  // namespace split8
}  // namespace sv
