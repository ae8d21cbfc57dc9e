// How paged attention's work is dealt to CTAs (host and device; the host side
// is what the tests drive).
//
// A unit is one 128-position chunk of one (sequence, row block, kv head): the
// row block is up to `tokens` of the sequence's new tokens (all query heads of
// the kv head), so that its rows fit the MMA's narrow side.  Sequence q has
// blocks * n_kv_heads pairs of `chunks` units each, pairs in (row block, kv
// head) order; a sequence with rows but no positions has one (empty) chunk, so
// that its rows are written.  first[q] is the exclusive sum of the units, T their
// number.  Of C = min(CTAs, T) working CTAs, CTA c takes the contiguous units
// [T c / C, T (c+1) / C): at least one, and every CTA the same number give or
// take one, whatever the lengths are.
//
// A maximal run of one pair's units inside a CTA is a segment.  A segment that
// covers its pair writes the rows' results; any other leaves a partial
// (unnormalised output, running maximum and sum) in slot 2c when it begins the
// CTA's range and in slot 2c+1 otherwise (then it ends the range).  The CTA
// where a split pair begins is its owner; the partials of a pair are the owner's
// and the first slots of the CTAs after it up to the pair's last unit.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define SPLIT_HD __host__ __device__ __forceinline__
#else
#define SPLIT_HD inline
#endif

namespace sv {
namespace split {

constexpr int kChunk = 128;          // positions per unit
constexpr int kMaxSeqs = 1024;

// Units of a sequence (its rows and length already checked).
SPLIT_HD int chunks_of(int len) { return len > 0 ? (len - 1) / kChunk + 1 : 1; }
SPLIT_HD int blocks_of(int rows, int tokens) { return rows > 0 ? (rows - 1) / tokens + 1 : 0; }
SPLIT_HD int64_t units_of(int rows, int len, int tokens, int hkv) {
    return (int64_t)blocks_of(rows, tokens) * hkv * chunks_of(len);
}

// CTAs that work on `total` units, and the first unit of the c-th.
SPLIT_HD int working(int ctas, int total) { return total < ctas ? total : ctas; }
SPLIT_HD int begin_of(int c, int total, int work) { return c < work ? (int)((int64_t)total * c / work) : total; }

// The CTA that works on unit u: the last c with begin_of(c) <= u.
SPLIT_HD int cta_of(int u, int total, int work) { return (int)((((int64_t)u + 1) * work - 1) / total); }

// The sequence that holds unit u < first[nseq]: the last q with first[q] <= u.
SPLIT_HD int sequence_of(const int* first, int nseq, int u) {
    int lo = 0, hi = nseq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= u) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Number of partials of a pair whose units end at pair_end (exclusive), owner c included.
SPLIT_HD int contributors(int c, int pair_end, int total, int work) { return cta_of(pair_end - 1, total, work) - c + 1; }

// Tile height (rows per kv head) for blocks of max_new tokens of G query
// heads: the smallest of 16, 32, 64, 128 that holds a whole block, else 128.
SPLIT_HD int tile_rows(int group, int max_new) {
    const int64_t want = (int64_t)group * max_new;
    return want <= 16 ? 16 : want <= 32 ? 32 : want <= 64 ? 64 : 128;
}

}  // namespace split
}  // namespace sv
