// How paged attention's work is dealt to CTAs (host and device; the host side
// is what the tests drive).
//
// A unit is one 128-position chunk of one (sequence, row block, kv head): the
// row block is up to `tokens` of the sequence's new tokens (all query heads of
// the kv head), so that its rows fit the MMA's narrow side.  Sequence q has
// blocks * n_kv_heads pairs of `chunks` units each, pairs in (row block, kv
// head) order; a sequence with rows but no positions has one (empty) chunk, so
// that its rows are written.  first[q] is the exclusive sum of the units, T their
// number.  C = min(CTAs, T) CTAs work, each on the same number of contiguous
// units give or take one, whatever the lengths are: the first T mod C CTAs take
// T / C + 1, the others T / C.
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

// The deal of `total` units to at most `ctas` CTAs.
struct Deal {
    int total, work, each, more;    // work CTAs; `more` of them take each + 1 units, the rest `each`
    SPLIT_HD Deal(int t, int ctas) : total(t), work(t < ctas ? t : ctas), each(work ? t / work : 0), more(t - each * work) {}
    // first unit of CTA c (the total from `work` on)
    SPLIT_HD int begin(int c) const { return c < work ? c * each + (c < more ? c : more) : total; }
    // the CTA that works on unit u < total
    SPLIT_HD int cta(int u) const { return u < more * (each + 1) ? u / (each + 1) : more + (u - more * (each + 1)) / each; }
    // partials of a pair that begins in CTA c and whose units end at pair_end (exclusive), c's included
    SPLIT_HD int parts(int c, int pair_end) const { return cta(pair_end - 1) - c + 1; }
};

// The sequence that holds unit u < first[nseq]: the last q with first[q] <= u.
SPLIT_HD int sequence_of(const int* first, int nseq, int u) {
    int lo = 0, hi = nseq;
#ifdef __CUDACC__
#pragma unroll 1
#endif
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= u) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Whether pairs are left whole: a CTA then takes the pairs that begin in its
// range, nothing is joined and no scratch is used.  Measured on the GPU, split
// against whole (8 kv heads of 128, decode, every sequence full): tables of 512
// positions 7.9 / 7.2 us with one sequence, 10.9 / 8.7 with 16, 28.3 / 26.3 with 64;
// 1024 positions 8.3 / 8.9, 13.1 / 10.8 and 47.8 / 45.6; 2048 positions 9.0 / 12.3,
// 27.6 / 24.8 and 85.2 / 83.6.  The caller also saves a launch and the scratch (4.3
// us of host time for a call against 7.0), so tables of up to 1024 positions stay whole.
SPLIT_HD bool whole_pairs(int table_pages) { return table_pages <= 16; }

// Tile height (rows per kv head) for blocks of max_new tokens of G query
// heads: the smallest of 16, 32, 64, 128 that holds a whole block, else 128.
SPLIT_HD int tile_rows(int group, int max_new) {
    const int64_t want = (int64_t)group * max_new;
    return want <= 16 ? 16 : want <= 32 ? 32 : want <= 64 ? 64 : 128;
}

}  // namespace split
}  // namespace sv
