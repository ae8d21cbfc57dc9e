// Shared memory of paged attention over an 8-bit cache (host and device; the host
// side is what the tests drive): what a CTA keeps in static memory, and how many
// tiles fit beside it.
#pragma once

#include <stdint.h>

#include "paged_plan.h"

namespace sv {
namespace plan8 {

using plan::kFewSeqs;
using plan::kSegs;
using plan::kSmem;
using plan::kWarps;
using plan::Pair;
using plan::Seg;
using split::kChunk;

constexpr int kSlots = 8;                   // at most, of K and of V
constexpr int kScaleSlots = 8;              // chunks whose scales are loaded ahead
constexpr int kParts = 3;                   // parts of a weight

// Tile height of a plan: which warpgroups work how, and how many buffers they take.
template <int RP>
struct Rows {
    static constexpr bool kStream = RP <= 64;               // warpgroups take alternate chunks
    static constexpr bool kStack = RP <= 32;                // P^T's parts in one product
    static constexpr int NQ = RP <= 64 ? 2 : 1;             // query tiles
    static constexpr int NP = kStream ? 2 : 1;              // P^T's
    static constexpr int kGroups = kStream ? 2 : 1;         // O^T's (and references) of a segment
};

// Everything but the tiles.
template <int RP>
struct Fixed {
    using T = Rows<RP>;
    alignas(16) uint8_t scale[kScaleSlots][2][2][64];   // of a chunk: by page, keys' and values'
    alignas(16) Seg segs[kSegs];
    alignas(16) float nref[2][T::kGroups][RP];      // by segment parity: minus each row's reference
    alignas(16) float qmul[2][RP];                  // by segment parity: log2 units per unit of S^T
    alignas(16) float xl[2][T::kGroups][4][RP];     // per lane quadrant: sums (and, while a reference moves, maxima)
    alignas(16) int tok[RP];                        // token of each row
    Pair weight[2][RP];                             // what the two O^T's of a row are multiplied with
    long long col_off[RP];                          // a row's offset in the output
    long long warp_sum[kWarps];
    uint64_t k_full[kSlots], k_empty[kSlots], v_full[kSlots], v_empty[kSlots], c_full[kScaleSlots], c_empty[kScaleSlots],
        q_full[T::NQ], q_empty[T::NQ], r_full[2], s_full[2], s_empty[2], p_full[T::NP], p_empty[T::NP], o_full[2], o_empty[2],
        l_full[2], l_empty[2], seg_full[kSegs], seg_empty[kSegs], fin[2];
    int first[split::kMaxSeqs + 1];
    int few_start[kFewSeqs + 1], few_len[kFewSeqs]; // a batch this small is not read from memory twice
    int vtop[2][4];                                 // by softmax warpgroup and quadrant: largest value scale of a chunk
    int vref[2][2];                                 // by segment parity and softmax warpgroup: the value scale that its weights are in
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
    static constexpr int kOther = T::NQ * kQ + T::NP * kParts * kP + 1024 + kPad;   // 1024: alignment
    static constexpr int kMost = kSmem - (int)sizeof(Fixed<RP>) - kOther;
    static constexpr int kFit = kMost / kSlot / 2;
    static constexpr int NK = kFit < kSlots ? kFit : kSlots, NV = NK;
    static constexpr int kBytes = kOther + (NK + NV) * kSlot;
    static constexpr int kO = T::kStack ? kParts * RP : RP; // tensor-memory columns of one O^T
    static constexpr int kUsed = 2 * RP + 2 * T::kGroups * kO;      // S^T x 2, O^T x 2 (per warpgroup)
    static constexpr int kCols = kUsed <= 256 ? 256 : 512;
    // registers of a thread, by role: 128 each at launch, moved to where S^T and P^T live
    static constexpr int kSoftRegs = RP <= 32 ? 160 : 184, kIssueRegs = 64, kResultRegs = RP <= 32 ? 128 : 80;
    static_assert(2 * kSoftRegs + kIssueRegs + kResultRegs <= 4 * 128, "more registers than the block was launched with");
    static_assert(NK >= 2 && kUsed <= 512, "a K and a V beyond those in use");
    static_assert(kBytes + (int)sizeof(Fixed<RP>) <= kSmem, "more shared memory than a CTA has");
};

}  // namespace plan8
}  // namespace sv
