// Shared memory of paged attention (host and device; the host side is what the
// tests drive): what a CTA keeps in static memory, and how many tiles fit beside it.
#pragma once

#include <stdint.h>

#include "paged_split.h"

namespace sv {
namespace plan {

using split::kChunk;

constexpr int kSmem = 227 * 1024;           // of a CTA
constexpr int kSlots = 8;                   // at most, of K and of V
constexpr int kSegs = 4;                    // segments listed ahead
constexpr int kFewSeqs = 64;                // a batch whose lengths are kept in shared memory
constexpr int kWarps = 16;

// Limits of one wait (2^31 cycles each) that the results of a segment are waited for.
// Other waits last a few chunks at most, this one all of them: up to 2^19, at 3000
// cycles each and 17000 at 128 rows where every chunk takes its scores again (364 us
// for 100003 positions against 94), more beside other kernels.
constexpr int wait_rounds(int units) { return 1 + (units >> 15); }

// A segment, as the roles need it.
struct alignas(16) Seg {
    int c0, units;              // first chunk, number of chunks (0: the list ends)
    int R;                      // rows
    int last0;                  // last position that the first token sees
    int len;                    // of the sequence
    int q, head;                // sequence, kv head
    int row0;                   // first row of the call
    int slot;                   // where its partial goes; -1: it covers its pair
    int pad[3];
};

struct alignas(8) Pair {
    float x, y;
};

// Tile height of a plan: which warpgroups work how, and how many buffers they take.
template <int RP>
struct Rows {
    static constexpr bool kStream = RP <= 64;               // warpgroups take alternate chunks
    static constexpr bool kStack = RP <= 32;                // P^T's parts in one product
    static constexpr int NQ = RP <= 32 ? 2 : 1;             // query tiles
    static constexpr int NP = kStream ? 2 : 1;              // pairs of P^T parts
    static constexpr int kGroups = kStream ? 2 : 1;         // O^T's (and references) of a segment
};

// Everything but the tiles.
template <int RP>
struct Fixed {
    using T = Rows<RP>;
    alignas(16) Seg segs[kSegs];
    alignas(16) float nref[2][T::kGroups][RP];      // by segment parity: minus each row's reference
    alignas(16) float xl[2][T::kGroups][4][RP];     // per lane quadrant: sums (and, while a reference moves, maxima)
    alignas(16) int tok[RP];                        // token of each row
    Pair weight[2][RP];                             // what the two O^T's of a row are multiplied with
    long long col_off[RP];                          // a row's offset in the output
    long long warp_sum[kWarps];
    uint64_t k_full[kSlots], k_empty[kSlots], v_full[kSlots], v_empty[kSlots], q_full[T::NQ], q_empty[T::NQ], s_full[2],
        s_empty[2], p_full[T::NP], p_empty[T::NP], o_full[2], o_empty[2], l_full[2], l_empty[2], seg_full[kSegs], seg_empty[kSegs],
        fin[2];
    int first[split::kMaxSeqs + 1];
    int few_start[kFewSeqs + 1], few_len[kFewSeqs]; // a batch this small is not read from memory twice
    int poison[2];                                  // 1 + the last segment (by parity) that silenced a value
    uint32_t tmem_base;
    int dead, total;
};

// NK slots for a chunk's K and NV for its V.  K and V do not share slots: different
// threads wait for them, and a barrier's parity is only sound for one that sees
// every phase.
template <int HD, int RP>
struct Plan : Rows<RP> {
    using T = Rows<RP>;
    static constexpr int kSlot = kChunk * HD * 2;
    static constexpr int kQ = RP * HD * 2;
    static constexpr int kP = kChunk * RP * 2;              // one part
    static constexpr int kOther = T::NQ * kQ + T::NP * 2 * kP + 2048;   // alignment, pad after the last slot
    static constexpr int kMost = kSmem - (int)sizeof(Fixed<RP>) - kOther;
    static constexpr int NS = kMost / kSlot < kSlots ? kMost / kSlot : kSlots;
    // V slots hold a chunk, or from 64 rows on, where there is room for few, a page:
    // the next chunk's first page then loads while this one's is still in use.
    // Of an odd number of pages K takes the rounded up half.
    static constexpr int kPieces = RP >= 64 ? 2 : 1, kPiece = kSlot / kPieces;
    static constexpr int NK = kPieces == 2 ? (kMost / kPiece + 2) / 4 : NS / 2;
    static constexpr int NV = (kMost - NK * kSlot) / kPiece < kSlots ? (kMost - NK * kSlot) / kPiece : kSlots;
    static constexpr int kBytes = kOther + NK * kSlot + NV * kPiece;
    static constexpr int kO = T::kStack ? 2 * RP : RP;      // tensor-memory columns of one O^T
    static constexpr int kUsed = 2 * RP + 2 * T::kGroups * kO;      // S^T x 2, O^T x 2 (per warpgroup)
    static constexpr int kCols = kUsed <= 256 ? 256 : 512;
    // registers of a thread, by role: 128 each at launch, moved to where S^T and P^T live
    static constexpr int kSoftRegs = RP <= 32 ? 160 : 184, kIssueRegs = 64, kResultRegs = RP <= 32 ? 128 : 80;
    static_assert(2 * kSoftRegs + kIssueRegs + kResultRegs <= 4 * 128, "more registers than the block was launched with");
    static_assert(NK >= 1 && NV >= kPieces + 1 && kUsed <= 512, "a K, and a V beyond the one in use");
    static_assert(NK <= kSlots && kBytes + (int)sizeof(Fixed<RP>) <= kSmem, "more shared memory than a CTA has");
};

}  // namespace plan
}  // namespace sv
