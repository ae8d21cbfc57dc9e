// Shared memory of paged attention over an 8-bit cache (host and device; the host
// side is what the tests drive): what a CTA keeps in static memory, and how many
// tiles fit beside it.
#pragma once

#include <stdint.h>

#include "paged_split8.h"

namespace sv {
namespace plan8 {

using split8::kChunk;

constexpr int kSmem = 227 * 1024;           // of a CTA
// K and V that a CTA has in flight or in use, 64 KB of each: 8 slots of 64-wide heads, 4
// of 128-wide ones, where there is room for 6, but 64 ragged decodes take 94.0 us with
// 6, 92.9 with 5, 91.7 with 4, 93.3 with 3 (of 64-wide ones fewer than 8 cost up to 15 %).
constexpr int kAhead = 64 * 1024;
constexpr int kSlots = kAhead / (kChunk * 64);
constexpr int kScaleSlots = 8;              // chunks whose scales are loaded ahead
constexpr int kParts = 3;                   // parts of a weight
// A row's largest contribution (weight times value scale) is kept at 2 to 4: a half overflows
// 2^14 above it, and small contributions end 1.5 * 2^-25 of it.  A bit more for these costs
// references that move: 24 sequences of 16 new at 8 heads a kv head 130.9 us with 2, 133.1 with
// 3, 136.5 with 4 (200 short ones 49.3, 50.3, 51.4).
constexpr int kShift8 = 2;
constexpr int kPart2 = 8, kPart3 = 16;      // the second part is kept times 8, the third times 8 * 16
constexpr int kSegs = 8;                    // segments in the list: those ahead, and those whose results are not written
constexpr int kFewSeqs = 64;                // a batch whose lengths are kept in shared memory

// Limits of one wait (2^31 cycles each) for what comes when a segment's chunks are through:
// the next entry of the list, which follows the last copy of K (the results' warps and softmax
// warps without rows wait for it from the segment's start), and the sums.  The other waits
// last a few chunks at most, these all of them, up to 2^19.
constexpr int wait_rounds(int units) { return 1 + (units >> 15); }

// A segment, as the roles need it.
struct alignas(16) Seg {
    int c0, units;              // first chunk, number of chunks (0: the list ends)
    int R;                      // rows
    int last0;                  // last position that the first row's token sees
    int len;                    // of the sequence
    int q, head;                // sequence, kv head
    int row0;                   // the first row's row of the call
    int skip;                   // query heads of that row in front of the first row
    int slot;                   // where its partial goes; -1: it covers its pair
    int pad[2];
};

struct alignas(16) Out {
    float f[2];                 // what the row is multiplied with in each team's O^T
    long long at;               // where the row goes, in elements behind the segment's first
};

// Tile height of a plan: how the softmax warpgroups share the work.  A thread handles
// one key and NC rows.
template <int RP>
struct Rows {
    static constexpr int NC = 16;                           // rows of a thread
    static constexpr int kSoftGroups = RP <= 16 ? 2 : 4;    // softmax warpgroups
    static constexpr int kTeam = RP / NC;                   // warpgroups of a chunk
    static constexpr bool kStream = kTeam < kSoftGroups;    // two teams take alternate chunks
    static constexpr int kGroups = kStream ? 2 : 1;         // O^T's (and references) of a segment
    static constexpr int NS = RP <= 32 ? 4 : 2;             // S^T's: two ahead of each team, where tensor memory has room
    static constexpr int kWarps = 4 * kSoftGroups + 8;
    static_assert(kTeam * kGroups == kSoftGroups, "every warpgroup has its share");
};

// Everything but the tiles.
template <int RP>
struct Fixed {
    using T = Rows<RP>;
    alignas(16) uint8_t scale[kScaleSlots][2][2][64];   // of a chunk: by page, keys' and values'
    alignas(16) Seg segs[kSegs];
    alignas(16) float nref[2][T::kGroups][RP];      // by segment parity: minus each row's reference
    alignas(16) float gain[2][T::kGroups][RP];      // and what its weights are multiplied with before their values' scales
    alignas(16) float qmul[2][RP];                  // by segment parity: log2 units per unit of S^T
    alignas(16) float shrink[T::kGroups][RP];       // while references move: what the old weights shrink by,
    alignas(16) float oshrink[T::kGroups][RP];      // and O^T, in which the gains are too
    alignas(16) float xl[2][T::kGroups][4][RP];     // per lane quadrant: sums (and, while a reference moves, maxima)
    alignas(16) float xc[T::kGroups][4][RP];        // while it moves: the largest contribution beside that maximum
    int top[T::kGroups][RP];                        // of each row: the exponent byte of its largest contribution so far
    alignas(16) int tok[RP];                        // token of each row of a block that begins with a token
    Out row[2][RP];                                 // by segment parity: for the results
    long long warp_sum[T::kWarps];
    uint64_t k_full[kSlots], k_empty[kSlots], v_full[kSlots], v_empty[kSlots], c_empty[kScaleSlots], q_full[2],
        q_empty[2], r_full[2], s_full[T::NS], s_empty[T::NS], p_full[2], p_empty[2], o_full[2], o_empty[2], l_full[2], l_empty[2],
        seg_full[kSegs], seg_empty[kSegs], fin[2];
    int first[split::kMaxSeqs + 1];
    int few_start[kFewSeqs + 1], few_len[kFewSeqs]; // a batch this small is not read from memory twice
    int tops[T::kSoftGroups][2];                       // by softmax warpgroup: its rows' largest contribution, and that of all if it is one
    int poison[2];                                  // 1 + the last segment (by parity) that silenced a value
    uint32_t tmem_base;
    int dead, total;
};

template <int HD, int RP>
struct Plan : Rows<RP> {
    using T = Rows<RP>;
    static constexpr int kSlot = kChunk * HD;               // a chunk's K or V
    static constexpr int kQPart = RP * HD;                  // one part of a query tile
    static constexpr int kQ = 2 * kQPart;
    static constexpr int kP = kChunk * RP;                  // one part of P^T
    static constexpr int kPad = 1024;                       // an M = 128 product over 64 dimensions reads past its slot
    static constexpr int kOther = 2 * kQ + 2 * kParts * kP + 1024 + kPad;   // two query tiles, two P^T's; 1024: alignment
    static constexpr int kMost = kSmem - (int)sizeof(Fixed<RP>) - kOther;
    static constexpr int kFit = kMost / kSlot / 2;
    static constexpr int NK = kFit < kAhead / kSlot ? kFit : kAhead / kSlot, NV = NK;
    static constexpr int kBytes = kOther + (NK + NV) * kSlot;
    static constexpr int kO = kParts * RP;                  // tensor-memory columns of one O^T: its parts side by side
    static constexpr int kUsed = T::NS * RP + 2 * T::kGroups * kO;  // S^T's, O^T x 2 (per team)
    static constexpr int kCols = kUsed <= 256 ? 256 : 512;
    // Registers of a thread, by role: the same for all at launch, moved to where S^T and P^T
    // live.  (Four softmax warpgroups leave 480 to share out: 88, 48 and 80 spill least
    // and take 24 sequences of 16 new at 8 heads a kv head from 127 us, with 88, 56 and 72, to 124.)
    static constexpr bool kTwo = T::kSoftGroups == 2;
    static constexpr int kLaunchRegs = kTwo ? 128 : 80, kSoftRegs = kTwo ? 160 : 88, kIssueRegs = kTwo ? 56 : 48, kResultRegs = kTwo ? 112 : 80;
    static_assert(T::kSoftGroups * kSoftRegs + kIssueRegs + kResultRegs <= (T::kSoftGroups + 2) * kLaunchRegs,
                  "more registers than the block was launched with");
    static_assert(T::kWarps * 32 * kLaunchRegs <= 65536, "more registers than an SM has");
    static_assert(NK >= 2 && kUsed <= 512, "a K and a V beyond those in use");
    static_assert(kBytes + (int)sizeof(Fixed<RP>) <= kSmem, "more shared memory than a CTA has");
};

}  // namespace plan8
}  // namespace sv
