// Attention of each sequence's newest positions over the 8-bit paged cache, on the
// fifth-generation tensor cores with the codes as they lie.
//
// The pipeline is that of the bf16 pages' attention (keys and head dimensions along
// the 128 tensor-memory lanes, query rows on the narrow side, one role a warp or
// warpgroup, chunks of 128 positions dealt evenly to CTAs); what differs is how 8 bits
// meet 16.  Per chunk:
//     S^T = K8 Q^T      K8: e4m3 codes.  q = 2^a (q1 + q2), two e4m3 parts with a power
//                       of two for each row: bf16's 8 significant bits are two times
//                       e4m3's 4 (the second part carries a sign), so that nothing of
//                       q is lost but below 2^-17 of the row's largest element.  The
//                       parts are two products into the same S^T.
//     P^T = exp2(2^(a + ek) scale log2e S^T - m)    ek: the key's scale
//     O^T += V8^T P'^T  P' = g 2^ev P as a half, in three e5m2 parts; ev: the value's scale
// A value's scale goes into its weight, so that the codes enter the product as they are.
// The row's gain g, a power of two, brings the largest contribution P 2^ev among the keys
// that the row sees to 2 .. 4: what counts is what a position adds to the result, so that
// a value that the row does not see or gives next to no weight sets nothing, however large it is,
// and neither does a key that takes all weight and has no value.  (The sums are of P, in 32
// bits; the results divide by g.)  Weights need more range than bits
// (a key far down still counts when there are 100000 like it), so their parts are
// e5m2, a half's upper byte: 3 significant bits each, which is cheap to round a half to
// (an addition, an and, a subtraction, a byte permutation).  What a part leaves is at most
// half of its last bit, so that it can be kept times 8, then times 16 more, without passing
// the weight: off by 2^-11 of the weight's power of two (and 2^-11 by the half), and by
// 2^-24 where e5m2 and halves end (2^-17 / 128, and 2^-25), 1.5 * 2^-25 of the largest
// contribution.  (Parts that are cut and kept times 4 and 8 left 2^-10 and 2^-22; 24 sequences of
// 16 new at 8 heads a kv head took 125.4 us with them, 128.8 so.)  A NaN may get lost in the
// parts, not in its row's sum, by which the row is divided.  The parts
// lie side by side in the product's N (3 RP columns of O^T, joined by the results): one
// product for all costs as much as one part's as long as N is this small.
//
// The 16 rows of a thread whose largest contributions lie within 2^3 of one another, as rows
// of one size of values do, share the largest's gain, which then is one factor a key: a
// multiplication for every two weights less (the same case 139 us without sharing, 131 with).
// It costs the smallest of them 3 bits at the lower end.
//
// A half's first part overflows 2^14 above the references.  So a segment's first chunk gives
// them (by row, the largest score and contribution), and a later chunk in which some half
// overflows makes its warpgroup move references, gains, sums and O^T up to its own, and is
// taken again; the vote on it rides on the barrier that the P^T buffer needs anyway.
//
// Roles, by warpgroup: softmax (thread = key, 16 rows; 2 of them for tiles of 16 rows,
// which take alternate chunks, else 4: two teams of 2, or one of 4); then one warp each
// for the MMAs of S^T, those of O^T, the copies of V, and the list of segments with the
// copies of K and the scales; last a warpgroup that splits the next segment's queries
// into their parts, then writes this segment's results (thread = head dimension).
// 16 rows a thread in 4 warpgroups took what 32 rows in 2 did (24 sequences of 16 new at
// 8 heads a kv head: 206 against 210 us then, 200 short ones 62 and 62), and one code
// serves every tile.
//
// What bounds it: long caches memory (100003 positions of 8 kv heads of 128: 39.9 us, 30.3
// at the copy rate; 64 ragged decodes 91.1, of 83), short sequences a segment's way through
// the roles (2.2 us a segment of one chunk at 16 rows, 0.4 a further chunk of 64-wide
// heads; 200 ragged blocks 49.6 us), many rows a chunk's way through the softmax (64 rows:
// about 2300 cycles, half of them issue; 24 sequences of 16 new at 8 heads a kv head 131 us).
// The roles share one instruction cache, so that code costs time wherever it stands: the
// last two were 62 and 154 us when the kernel had 86 KB (46 and 124 with 71), with divisions in
// the walk over the segments, each wait's loop twice, and rows' addresses formed where they are written.
#include <stddef.h>
#include <stdio.h>

#include "paged_core.cuh"
#include "paged_plan8.h"

namespace sv {
namespace {

using plan8::kFewSeqs;
using plan8::kPart2;
using plan8::kPart3;
using plan8::kParts;
using plan8::kScaleSlots;
using plan8::kSegs;
using plan8::kShift8;
using plan8::Plan;
using plan8::Seg;

// A row's largest contribution (weight times value scale) is kept as an exponent byte, top;
// its gain is 2^(kShift8 + 127 - top).
constexpr int kGainBytes = 254 + kShift8;   // exponent byte of a gain, plus top
constexpr int kLeastTop = 1 + kShift8;      // the gain stays below 2^127
constexpr int kSpread = 3;                  // rows of a thread whose tops lie this close share the largest
constexpr int kMostBytes = 127 - kShift8;   // a value scale further above a shared top has no factor
constexpr int kApart = -512;                // (in place of one: rows that share none)
constexpr int kFarScale = 40;               // a value scale this far below every top: its weight overflows no half before sums might,
constexpr float kFarWeight = 1ull << (16 - kShift8 + kFarScale);    // so it is looked at itself (one that halves let pass is no larger)

struct Paged8Params : PagedCommon {
    CUtensorMap mk, mv;
    int tile;                   // rows of a block
    const uint16_t* q;
    long long q_stride;
    const uint8_t *vpool, *scales;
};

// Barriers and shared memory by 32-bit addresses: the roles' loops are short enough for
// a conversion per access to be much of what they do.  `kept` makes a value stay in its
// register: a shared address is otherwise formed anew wherever it is used.
__device__ __forceinline__ uint32_t kept(uint32_t v) {
    asm volatile("mov.b32 %0, %0;" : "+r"(v));
    return v;
}
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}
// The word at `dead`, which a wait that gave up sets.
__device__ __forceinline__ bool raised(uint32_t dead) {
    uint32_t v;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(dead) : "memory");
    return v != 0;
}
__device__ __forceinline__ void raise(uint32_t dead) { asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(dead), "r"(1u) : "memory"); }
// Wait bounded in time (2^31 cycles, about a second, `rounds` of them): one that gives
// up raises dead, and no wait lasts once that is raised.  For whole warps: a try by
// part of a warp does not suspend it, and a spinning warp takes its neighbours' turns.
// The lanes may leave it apart: they join (__syncwarp, a vote, a named barrier) before
// one of them does what lets the barrier's next phase end, or the others could look after
// that, and wait for a phase that is over.  (Joining in here costs 1 to 5 %.)
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, uint32_t dead, int rounds = 1) {
    uint32_t t0 = cycles();
#pragma unroll 1
    while (!try_wait(bar, parity)) {
        if (raised(dead)) return false;
        if (cycles() - t0 > 0x7fffffffu) {
            if (--rounds <= 0) raise(dead);
            t0 = cycles();
        }
    }
    return true;
}
__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void arrive_if(uint32_t bar, bool one) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar), "r"((uint32_t)one) : "memory");
}
__device__ __forceinline__ void arrive_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void give_up(uint32_t bar, uint32_t parity) {  // after a failed wait: let what is in flight finish
#pragma unroll 1
    for (uint32_t i = 0; i < (1u << 20) && !try_wait(bar, parity); ++i) __nanosleep(64);
}
__device__ __forceinline__ void tile_load(uint32_t dst, const CUtensorMap* map, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(0), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ int lds_u8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return (int)v;
}
__device__ __forceinline__ float4 lds4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// D[tmem] (+)= A B^T in 8-bit floats, descriptors in halves.
__device__ __forceinline__ void umma8_lo(uint32_t d, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Instruction descriptor of kind::f8f6f4 with fp32 D: formats 0 e4m3, 1 e5m2.
__host__ __device__ constexpr uint32_t idesc8(uint32_t m, uint32_t n, uint32_t a, uint32_t b) {
    return (1u << 4) | (a << 7) | (b << 10) | ((n >> 3) << 17) | ((m >> 4) << 24);
}
// Halves of a matrix descriptor; a row of HD codes is the swizzle's width: 128 or 64 bytes.
template <int HD>
constexpr uint32_t hi_swizzled(uint32_t sbo) { return (sbo >> 4) | (1u << 14) | ((HD == 128 ? 2u : 4u) << 29); }
__device__ __forceinline__ uint32_t lo_desc(uint32_t saddr, uint32_t lbo) { return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16); }

// Where byte b (a multiple of 8) of row r lies in a swizzled tile of HD-byte rows.
template <int HD>
__device__ __forceinline__ int swizzled(int r, int b) {
    return HD == 128 ? r * 128 + ((((b >> 4) ^ r) & 7) << 4) + (b & 15) : r * 64 + ((((b >> 4) ^ (r >> 1)) & 3) << 4) + (b & 15);
}

// 2^(byte - 127)
__device__ __forceinline__ float scale_of(int byte) { return __uint_as_float(byte ? (uint32_t)byte << 23 : 1u << 22); }

__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Largest of the warp's values; a NaN counts only among NaN.
__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// Two floats' e4m3 codes (a in the low byte), and what they leave.
__device__ __forceinline__ uint32_t split_e4m3(float& a, float& b) {
    uint16_t c;
    uint32_t h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(b), "f"(a));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    float x, y;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}" : "=f"(x), "=f"(y) : "r"(h));
    a -= x;
    b -= y;
    return c;
}
// Halves: an e5m2 code is a half's upper byte.
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b) {    // a NaN counts only among NaN
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
constexpr uint32_t kHalves2 = 0x48004800u, kHalves3 = 0x4C004C00u;  // kPart2 and kPart3 twice
static_assert(kPart2 == 8 && kPart3 == 16, "as halves");
__device__ __forceinline__ uint32_t upper_bytes(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, 0x7531;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t cvt_f16x2(F2 x) {
    float a, b;
    x.get(a, b);
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// A CTA's segments in order.
struct Walk {
    const Paged8Params& p;
    const int* first;           // [nseq + 1] in shared memory
    const int *start, *lens;    // row starts and lengths: in shared memory when they are few
    int u, end;                 // next unit, end of the CTA's range
    int q = 0, q1 = 0;          // sequence, the end of its units
    int rows = 0, len = 0, row_base = 0, chunks = 1;
    // the segment
    int head = 0, c0 = 0, c1 = 0, seg = -1;
    int pair0 = 0;              // first unit of its pair
    split8::Place at = {0, 0};  // where its block begins

    __device__ Walk(const Paged8Params& pp, const int* f, const int* s, const int* n, int begin, int e)
        : p(pp), first(f), start(s), lens(n), u(begin), end(e) {}
    __device__ __forceinline__ void sequence() {
        q1 = first[q + 1];
        row_base = start[q];
        rows = start[q + 1] - row_base;
        len = lens[q];
        chunks = split8::chunks_of(len);
    }
    __device__ __forceinline__ bool next() {
#pragma unroll 1
        for (;;) {
            if (u >= end) return false;
            int u0 = 0;                             // the pair's first unit in the range
            if (q1 == 0) {                          // where the range begins
                q = split::sequence_of(first, p.nseq, u);
                sequence();
                const unsigned span = chunks + split8::kHead, v = u - first[q], pair = v / span, block = pair / (unsigned)p.hkv;
                head = pair - block * p.hkv;
                u0 = v - pair * span;
                at.at(block, p.group, p.tokens);
            } else {
                step();
            }
            pair0 = u - u0;
            const int span = chunks + split8::kHead, u1 = p.whole ? span : min(span, u0 + end - u);
            u += u1 - u0;
            if (p.whole && u0 > 0) continue;        // it begins in another CTA's range, which takes it
            const split8::Part part = split8::part_of(u0, u1);
            c0 = part.c0;
            c1 = part.c1;
            if (c1 > c0) break;                     // (else not one of its chunks lies in the range)
        }
        ++seg;
        return true;
    }
    // the pair after the current one
    __device__ __forceinline__ void step() {
        if (u >= q1) {
            do ++q;
            while (first[q + 1] <= u);              // sequences without units
            sequence();
            at = {0, 0};
            head = 0;
        } else if (++head == p.hkv) {
            head = 0;
            at.step(p.group, p.tokens);
        }
    }
    __device__ __forceinline__ bool whole() const { return c0 == 0 && c1 == chunks; }
    __device__ __forceinline__ Seg segment() const {
        Seg s = {};
        s.c0 = c0;
        s.units = c1 - c0;
        s.R = min(p.tile, min(rows - at.token, p.tile) * p.group - at.skip);
        s.last0 = len - rows + at.token;
        s.len = len;
        s.q = q;
        s.head = head;
        s.row0 = row_base + at.token;
        s.skip = at.skip;
        s.slot = whole() ? -1 : 2 * (int)blockIdx.x + (c0 > 0 ? 0 : 1);
        return s;
    }
    // the segment's pair, for the join
    __device__ __forceinline__ Meta meta(const split::Deal& deal, const Seg& s) const {
        Meta m;
        m.owner = split8::owner_of(deal, pair0);
        m.count = split8::parts_of(deal, m.owner, pair0, chunks);
        m.slot = 2 * m.owner + 1;
        m.rows = s.R;
        m.head = head * p.group;
        m.row0 = s.row0;
        m.last0 = s.last0;
        m.skip = s.skip;
        return m;
    }
};

template <int HD, int RP>
__global__ void __block_size__((32 * Plan<HD, RP>::kWarps, 1, 1)) __maxnreg__((Plan<HD, RP>::kLaunchRegs)) paged_attn8_kernel(const __grid_constant__ Paged8Params p) {
    using L = Plan<HD, RP>;
    constexpr bool kStream = L::kStream;
    constexpr int NK = L::NK, NV = L::NV, NS = L::NS, NC = L::NC;
    constexpr int kGroups = L::kGroups, kTeam = L::kTeam;
    constexpr int kArrive = kTeam;              // warpgroups that read an S^T and write a P^T
    constexpr int kThreads = 32 * L::kWarps, kSoftWarps = 4 * L::kSoftGroups;
    constexpr int kScoreWarp = kSoftWarps, kLoadVWarp = kScoreWarp + 2, kLoadKWarp = kScoreWarp + 3, kResultWarp = kScoreWarp + 4;
    constexpr int kReaders = kSoftWarps + 3 + 4;    // warps that read the list of segments
    constexpr int kSoftBar = 1, kResultBar = kSoftBar + L::kSoftGroups;     // named barriers: one per softmax warpgroup, the results' warpgroup
    extern __shared__ uint8_t smem_raw[];
    __shared__ plan8::Fixed<RP> sh;

    uint8_t* base = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* kslots = base;
    uint8_t* vslots = kslots + NK * L::kSlot;
    uint8_t* qs = vslots + NV * L::kSlot + L::kPad;
    uint8_t* ps = qs + 2 * L::kQ;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid < 32) {                             // the lanes share the barriers
        if (lane < NK) {
            mbar_init(&sh.k_full[lane], 1);
            mbar_init(&sh.k_empty[lane], 1);
        }
        if (lane < NV) {
            mbar_init(&sh.v_full[lane], 1);
            mbar_init(&sh.v_empty[lane], 1);
        }
        if (lane < NS) {
            mbar_init(&sh.s_full[lane], 2);     // the product, and the warp that saw its K's scales arrive
            mbar_init(&sh.s_empty[lane], kArrive);
        }
        if (lane < kScaleSlots) mbar_init(&sh.c_empty[lane], kArrive);
        if (lane < 2) {
            mbar_init(&sh.q_full[lane], 4);
            mbar_init(&sh.q_empty[lane], 1);
            mbar_init(&sh.r_full[lane], 4);
            mbar_init(&sh.o_full[lane], 1);
            mbar_init(&sh.o_empty[lane], 4);
            mbar_init(&sh.l_full[lane], kSoftWarps);
            mbar_init(&sh.l_empty[lane], 4);
            mbar_init(&sh.p_full[lane], kArrive);
            mbar_init(&sh.p_empty[lane], 1);
            mbar_init(&sh.fin[lane], 1);
            sh.poison[lane] = 0;
        }
        if (lane < kSegs) {
            mbar_init(&sh.seg_full[lane], 1);
            mbar_init(&sh.seg_empty[lane], kReaders);
        }
        fence_barrier_init();
        if (lane == 0) {
            sh.dead = 0;
            sh.first[0] = 0;
        }
    }
#pragma unroll 1
    for (int i = tid; i < RP; i += kThreads) sh.tok[i] = i / p.group;
    if (warp == kScoreWarp) tmem_alloc(&sh.tmem_base, L::kCols);
    pdl_wait();
    pdl_launch_dependents();

    // first[q]: exclusive sums of the sequences' units, 2 sequences a thread
    {
        static_assert(2 * kThreads >= split::kMaxSeqs, "2 sequences a thread");
        long long v[2], sum = 0;   // 64 bits: row ranges that overlap can pass any bound
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int q = tid * 2 + k;
            v[k] = 0;
            if (q < p.nseq) {
                const int r0 = p.row_start[q], r1 = p.row_start[q + 1], n = p.len[q];
                const bool bad_rows = r0 < 0 || r1 < r0 || r1 > p.rows;
                const bool bad_len = n < 0 || n > (long long)p.table_pages * SPEC_PAGE;
                if (p.nseq <= kFewSeqs) {
                    sh.few_start[q] = r0;
                    sh.few_start[q + 1] = r1;   // the next sequence's r0, the same word
                    sh.few_len[q] = n;
                }
                if (bad_rows || bad_len) {
                    if (blockIdx.x == 0 && p.err) atomicCAS(p.err, 0, bad_rows ? SPEC_PAGED_BAD_ROWS : SPEC_PAGED_BAD_LENGTH);
                } else {
                    v[k] = split8::units_of(r1 - r0, n, p.group, p.tokens, p.hkv);
                }
            }
            sum += v[k];
        }
        long long inc = sum;
#pragma unroll 1
        for (int d = 1; d < 32 && 2 * d < p.nseq; d <<= 1) {   // as far as there are sequences
            const long long o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        long long run = inc - sum;
        if (p.nseq > 64) {                      // more than one warp holds sequences
            if (lane == 31) sh.warp_sum[warp] = inc;
            __syncthreads();
#pragma unroll 1
            for (int w = 0; w < warp && w * 64 < p.nseq; ++w) run += sh.warp_sum[w];
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            run += v[k];
            if (tid * 2 + k < p.nseq) sh.first[tid * 2 + k + 1] = (int)run;
        }
        if (tid == (p.nseq - 1) / 2) {
            sh.total = run > 0x7fffffff ? 0 : (int)run;
            if (run > 0x7fffffff && blockIdx.x == 0 && p.err) atomicCAS(p.err, 0, SPEC_PAGED_BAD_ROWS);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    const split::Deal deal(sh.total, gridDim.x);
    const int begin = deal.begin(blockIdx.x), end = deal.begin(blockIdx.x + 1);
    // shared memory by address: barrier i of an array of them is BAR(array, i)
    using F = plan8::Fixed<RP>;
    const uint32_t shb = kept(smem_u32(&sh));
#define BAR(x, i) (shb + (uint32_t)offsetof(F, x) + (uint32_t)(i) * 8u)
    const uint32_t dead = shb + (uint32_t)offsetof(F, dead);
    // token of row r of a block, counted from its first row's (which the block may begin in the middle of)
    auto token = [&](const Seg& s, int r) { return RP == split8::kMostRows && p.group > RP ? (int)(s.skip + r >= p.group) : sh.tok[r]; };
    Ring<kSegs> sr;                             // every role's place in the list of segments
    int before = 0;                             // chunks of the segment before: who has no part in them waits here for all
    auto take = [&]() {                         // the next segment
        wait(BAR(seg_full, sr.at), sr.round, dead, plan8::wait_rounds(before));
        const Seg s = sh.segs[sr.at];
        before = s.units;
        __syncwarp();
        arrive_if(BAR(seg_empty, sr.at), lane == 0);
        sr.step();
        return s;
    };

    if (warp >= kScoreWarp && warp < kResultWarp) {
        regs_down<L::kIssueRegs>();
        if (warp == kLoadKWarp) {
            // ---------------- the list of segments, K and scale copies, and what the join kernel has to do here ----------------
            const bool few = p.nseq <= kFewSeqs;
            Walk w(p, sh.first, few ? sh.few_start : p.row_start, few ? sh.few_len : p.len, begin, end);
            Meta* const meta = p.meta + 2 * blockIdx.x;     // of the pair that goes on here, and of the one that goes on behind
            if (lane == 0 && !p.whole) meta[0] = meta[1] = {};
            Ring<NK> kr;
            Ring<kScaleSlots> cr;
            const uint32_t ka = kept(smem_u32(kslots));
            bool ok = true;
#pragma unroll 1
            for (bool more = true; more && ok;) {
                more = w.next();
                Seg s = {};                     // no units: the list ends
                if (more) {
                    s = w.segment();
                    if (lane == 0 && !p.whole && !w.whole()) meta[w.c0 == 0] = w.meta(deal, s);
                }
                ok = wait(BAR(seg_empty, sr.at), sr.round ^ 1, dead);
                if (!__all_sync(0xffffffffu, ok)) break;
                if (lane == 0) {
                    sh.segs[sr.at] = s;
                    arrive(BAR(seg_full, sr.at));
                }
                sr.step();
                if (!more) break;
                PageWalk pages;
#pragma unroll 1
                for (int k = 0; k < s.units; ++k) {
                    pages.at(p, s, k, lane);
                    ok = wait(BAR(c_empty, cr.at), cr.round ^ 1, dead);
                    ok = wait(BAR(k_empty, kr.at), kr.round ^ 1, dead) && ok;
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (elect_one()) {
                        const uint32_t full = BAR(k_full, kr.at);    // of K and its scales
                        const uint32_t to = shb + (uint32_t)offsetof(F, scale) + cr.at * 4 * SPEC_PAGE, dst = ka + kr.at * L::kSlot;
                        // a bad page (it reads as zeros) has no scales: ones
                        const bool c0 = pages.count > 0 && pages.z0 >= 0, c1 = pages.count > 1 && pages.z1 >= 0;
                        constexpr uint32_t kOnes = 0x7F7F7F7Fu;
                        if ((pages.count > 0 && !c0) || (pages.count > 1 && !c1)) {
#pragma unroll 1
                            for (int i = 0; i < 16; ++i)
                                if (i < 8 ? !c0 : !c1) sts4(to + i * 16, kOnes, kOnes, kOnes, kOnes);
                            fence_proxy_async_smem();
                        }
                        arrive_expect_tx(full, (uint32_t)(pages.count * SPEC_PAGE * HD) + (c0 ? 2 * SPEC_PAGE : 0) + (c1 ? 2 * SPEC_PAGE : 0));
                        if (c0) bulk_load(to, p.scales + (size_t)pages.z0 * 2 * SPEC_PAGE, 2 * SPEC_PAGE, full);
                        if (c1) bulk_load(to + 2 * SPEC_PAGE, p.scales + (size_t)pages.z1 * 2 * SPEC_PAGE, 2 * SPEC_PAGE, full);
                        if (pages.count > 0) tile_load(dst, &p.mk, pages.z0, full);
                        if (pages.count > 1) tile_load(dst + SPEC_PAGE * HD, &p.mk, pages.z1, full);
                    }
                    __syncwarp();
                    kr.step();
                    cr.step();
                }
            }
            if (lane == 0 && raised(dead)) {          // every buffer's last copy, as far as one was issued
#pragma unroll 1
                for (int i = 0; i < NK; ++i) give_up(BAR(k_full, i), i < kr.at ? kr.round : kr.round ^ 1);
            }
        } else if (warp == kLoadVWarp) {
            // ---------------- V copies ----------------
            Ring<NV> vr;
            const uint32_t va = kept(smem_u32(vslots));
            bool ok = true;
#pragma unroll 1
            for (;;) {
                const Seg s = take();
                ok = __all_sync(0xffffffffu, !raised(dead));
                if (!ok || s.units == 0) break;
                PageWalk pages;
#pragma unroll 1
                for (int k = 0; k < s.units; ++k) {
                    pages.at(p, s, k, lane);
                    ok = wait(BAR(v_empty, vr.at), vr.round ^ 1, dead);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (elect_one()) {
                        const uint32_t full = BAR(v_full, vr.at), dst = va + vr.at * L::kSlot;
                        arrive_expect_tx(full, (uint32_t)(pages.count * SPEC_PAGE * HD));
                        if (pages.count > 0) tile_load(dst, &p.mv, pages.z0, full);
                        if (pages.count > 1) tile_load(dst + SPEC_PAGE * HD, &p.mv, pages.z1, full);
                    }
                    __syncwarp();
                    vr.step();
                }
                if (!ok) break;
            }
            if (lane == 0 && raised(dead)) {
#pragma unroll 1
                for (int i = 0; i < NV; ++i) give_up(BAR(v_full, i), i < vr.at ? vr.round : vr.round ^ 1);
            }
        } else if (warp == kScoreWarp) {
            // ---------------- MMAs of S^T (the warp waits, one elected thread issues) ----------------
            Ring<NK> ks;
            Ring<2> qr;
            Ring<NS> sb;
            const uint32_t sa = kept(smem_u32(kslots)), qa = kept(smem_u32(qs));
            bool ok = true;
#pragma unroll 1
            while (ok) {
                const Seg s = take();
                ok = __all_sync(0xffffffffu, !raised(dead));
                if (!ok || s.units == 0) break;
                ok = wait(BAR(q_full, qr.at), qr.round, dead);
                const uint32_t id = idesc8(128, (s.R + 15) & ~15, 0, 0);
                const uint32_t dq = lo_desc(qa + qr.at * L::kQ, 16);
                constexpr uint32_t kHi = hi_swizzled<HD>(8 * HD);
#pragma unroll 1
                for (int k = 0; k < s.units; ++k) {
                    ok = wait(BAR(k_full, ks.at), ks.round, dead) && ok;
                    ok = wait(BAR(s_empty, sb.at), sb.round ^ 1, dead) && ok;
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t dk = lo_desc(sa + ks.at * L::kSlot, 16);
#pragma unroll
                        for (int part = 0; part < 2; ++part)
#pragma unroll
                            for (int e = 0; e < HD / 32; ++e)
                                umma8_lo(tmem + sb.at * RP, dk + e * 2, kHi, dq + part * (L::kQPart >> 4) + e * 2, kHi, id, (part | e) != 0);
                        commit(BAR(s_full, sb.at));
                        arrive(BAR(s_full, sb.at));             // (after K's barrier: the softmax reads scales that came with K)
                        commit(BAR(k_empty, ks.at));
                        if (k == s.units - 1) commit(BAR(q_empty, qr.at));
                    }
                    __syncwarp();
                    ks.step();
                    sb.step();
                }
                qr.step();
            }
            if (raised(dead)) {
                if (elect_one()) commit(BAR(fin, 0));
                __syncwarp();
                give_up(BAR(fin, 0), 0);
            }
        } else {
            // ---------------- MMAs of O^T (the same) ----------------
            Ring<NV> vs;
            Ring<2> pr;
            const uint32_t sa = kept(smem_u32(vslots)), pa = kept(smem_u32(ps));
            bool ok = true;
            int j = 0;                          // unit
#pragma unroll 1
            for (int seg = 0; ok; ++seg) {
                const Seg s = take();
                ok = __all_sync(0xffffffffu, !raised(dead));
                if (!ok || s.units == 0) break;
                ok = wait(BAR(o_empty, seg & 1), ((seg >> 1) & 1) ^ 1, dead);
                // A = V^T and B = P^T, both MN-major
                constexpr uint32_t id = idesc8(128, kParts * RP, 0, 1) | (1u << 15) | (1u << 16);
#pragma unroll 1
                for (int k = 0; k < s.units; ++k, ++j) {
                    ok = wait(BAR(v_full, vs.at), vs.round, dead) && ok;
                    ok = wait(BAR(p_full, pr.at), pr.round, dead) && ok;
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        // P^T: core matrices of 16 rows (of the product's N) x 8 keys, 128 bytes apart along the keys
                        const uint32_t dp = lo_desc(pa + pr.at * kParts * L::kP, 128);
                        const uint32_t dv = lo_desc(sa + vs.at * L::kSlot, 1024);
                        constexpr uint32_t kHiV = hi_swizzled<HD>(8 * HD), kHiP = (kChunk * 16 >> 4) | (1u << 14);
                        const int og = kStream ? (seg & 1) * 2 + (j & 1) : seg & 1;
                        const uint32_t o = tmem + NS * RP + og * L::kO;
                        const bool more = k >= kGroups;     // this O^T holds earlier chunks
#pragma unroll
                        for (int e = 0; e < kChunk / 32; ++e)
                            umma8_lo(o, dv + e * (32 * HD >> 4), kHiV, dp + e * (32 * 16 >> 4), kHiP, id, more || e != 0);
                        commit(BAR(v_empty, vs.at));
                        commit(BAR(p_empty, pr.at));
                        if (k == s.units - 1) commit(BAR(o_full, seg & 1));
                    }
                    __syncwarp();
                    vs.step();
                    pr.step();
                }
            }
            if (raised(dead)) {
                if (elect_one()) commit(BAR(fin, 1));
                __syncwarp();
                give_up(BAR(fin, 1), 0);
            }
        }
        __syncwarp();
    } else if (warp < kSoftWarps) {
        // ---------------- softmax: thread = key ----------------
        regs_up<L::kSoftRegs>();
        const int wg = warp >> 2, qd = warp & 3;
        const uint32_t lanes = kept(tmem + ((uint32_t)(qd * 32) << 16));
        const int key = qd * 32 + lane;
        const int gi = kStream ? wg / kTeam : 0;    // its team: which chunks, references and O^T
        const int col0 = (wg % kTeam) * NC;         // the thread's first row
        const int bar = kSoftBar + wg;
        const uint32_t scales = kept(shb + (uint32_t)offsetof(F, scale) + (key >> 6) * 2 * SPEC_PAGE + (key & 63));
        const uint32_t weights = kept(smem_u32(ps) + (col0 >> 4) * (kChunk * 16) + key * 16);
        uint32_t unit = 0;                      // the segment's first unit
#pragma unroll 1
        for (int seg = 0;; ++seg) {
            const Seg w = take();
            if (bar_any(bar, 128, raised(dead)) || w.units == 0) break;   // after a wait that gave up, all of the warpgroup leaves
            const int par = seg & 1, last0 = w.last0, rows = w.R - col0;   // live rows of this thread
            const int active = min((w.R + NC - 1) / NC, kTeam);     // warpgroups of the team with rows
            const bool speaks = key == 0;       // for the warpgroup
            const uint32_t mine = kept(shb + (uint32_t)offsetof(F, nref) + ((par * kGroups + gi) * RP + col0) * 4);
            const uint32_t qmul = kept(shb + (uint32_t)offsetof(F, qmul) + (par * RP + col0) * 4);
            wait(BAR(l_empty, par), ((seg >> 1) & 1) ^ 1, dead);     // the results of two segments ago have been read
            wait(BAR(r_full, par), (seg >> 1) & 1, dead);            // the query rows' powers of two are there
            F2 l[NC / 2];                       // the rows' sums over this thread's keys
#pragma unroll
            for (int j = 0; j < NC / 2; ++j) l[j] = F2(0.f, 0.f);
            const uint32_t gains = kept(shb + (uint32_t)offsetof(F, gain) + ((par * kGroups + gi) * RP + col0) * 4);
            bool fresh = true;
            int most = 0, shared = 0;           // the rows' largest top, and the one that they share
#pragma unroll 1
            for (uint32_t i = unit + (kStream ? (unit ^ gi) & 1u : 0u); i < unit + w.units; i += kGroups) {
                const uint32_t b = i & 1, use = (i >> 1) & 1;       // P^T buffer, its round
                if (rows <= 0) {
                    // No rows here: one warp keeps up with the team's barriers (a barrier's
                    // parity is only sound for one that sees every phase).
                    if (qd == 0) {
                        wait(BAR(s_full, i % NS), (i / NS) & 1, dead);
                        __syncwarp();
                        arrive_if(BAR(s_empty, i % NS), speaks);
                        arrive_if(BAR(c_empty, i % kScaleSlots), speaks);
                        wait(BAR(p_empty, b), use ^ 1, dead);
                        __syncwarp();
                        arrive_if(BAR(p_full, b), speaks);
                    }
                    continue;
                }
                const uint32_t st = lanes + i % NS * RP + col0;
                const int kp = (w.c0 + (int)(i - unit)) * kChunk + key;
                const bool masked = kp - key + kChunk - 1 > last0;  // some row does not see all of the chunk
                // One warp waits for the warpgroup.
                if (qd == 0) {
                    wait(BAR(s_full, i % NS), (i / NS) & 1, dead);
                    if (!kStream) wait(BAR(p_empty, b), use ^ 1, dead);
                }
                named_bar_sync(bar, 128);
                tc_fence_after();
                // the key's scales; NaN ones make its visible scores NaN, behind the length they are whatever stands there
                const uint32_t sc = scales + i % kScaleSlots * 4 * SPEC_PAGE;
                int vb = 0;
                float x[NC];                    // the rows' scores, then weights
#pragma unroll 1
                for (bool move = fresh;; move = true) {
                    tmem_ld16_async(st, x);
                    const int kb = lds_u8(sc);
                    vb = lds_u8(sc + SPEC_PAGE);
                    const float km = max(kb, vb) == 255 ? __uint_as_float(0x7FC00000u) : scale_of(kb);
                    if (vb == 255 || kp >= w.len) vb = 0;
                    const F2 km2(km, km);
                    // rows are in token order: the key is hidden from the tokens before it
                    const int hidden = min(max(kp - last0, 0), RP) * p.group - w.skip - col0;
                    tmem_wait_ld();
                    if (move) {
                        // The references move up to the chunk's maxima (a first chunk's become
                        // them), the sums and O^T with them.
                        float (*const mx)[RP] = sh.xl[par][gi], (*const cx)[RP] = sh.xc[gi];
                        const float ev = (float)vb;
#pragma unroll 1
                        for (int j = 0; j < NC && j < rows; j += 8) {
                            float v[8], m[8], keep = 0.f, keep2 = 0.f;
                            tmem_ld8_async(st + j, v);
                            const float4 f = lds4(qmul + j * 4), g = lds4(qmul + j * 4 + 16);
                            const float fs[8] = {f.x, f.y, f.z, f.w, g.x, g.y, g.z, g.w};
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                v[e] = j + e < hidden ? -INFINITY : __fmul_rn(__fmul_rn(v[e], km), fs[e]);
                                m[e] = warp_max(v[e]);
                                if (lane == e) keep = m[e];
                            }
                            // Contributions, beside the warp's largest weight: a difference of scores is
                            // exact where it counts, whatever their size.
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float c = warp_max(v[e] - m[e] + ev);
                                if (lane == e) keep2 = c;
                            }
                            if (lane < 8) mx[qd][col0 + j + lane] = keep, cx[qd][col0 + j + lane] = keep2;
                        }
                        // the last product into this O^T: of this team's chunk before
                        if (!fresh && qd == 0) wait(BAR(p_empty, (i - kGroups) & 1), ((i - kGroups) >> 1) & 1, dead);
                        named_bar_sync(bar, 128);
                        tc_fence_after();
                        if (key < NC) {         // one thread per row: the new reference, and what the old weights shrink by
                            const int r = col0 + key;
                            const bool live = key < rows;
                            const float m = fmaxf(fmaxf(mx[0][r], mx[1][r]), fmaxf(mx[2][r], mx[3][r]));
                            const float old = fresh ? kNone : -sh.nref[par][gi][r];
                            const float now = live ? fmaxf(old, m) : INFINITY;      // rows past R weigh nothing
                            sh.nref[par][gi][r] = -now;
                            // The largest contribution: this chunk's rounded up, the earlier ones' down.  (A row that
                            // sees nothing, or NaN alone, has none.)
                            const float c = fmaxf(fmaxf(cx[0][r] + (mx[0][r] - now), cx[1][r] + (mx[1][r] - now)),
                                                  fmaxf(cx[2][r] + (mx[2][r] - now), cx[3][r] + (mx[3][r] - now)));
                            const int old_top = fresh ? kLeastTop : sh.top[gi][r];
                            int top = max(max(__float2int_ru(c), __float2int_rd((float)old_top + (old - now))), kLeastTop);
                            sh.top[gi][r] = top;
                            const int was = fresh ? top : kGainBytes - (int)(__float_as_uint(sh.gain[par][gi][r]) >> 23);
                            const int high = __reduce_max_sync((1u << NC) - 1u, live ? top : 0);
                            // (one that has seen no key moves when it does)
                            const bool near = __all_sync((1u << NC) - 1u, !live || now == kNone || top >= high - kSpread);
                            if (near) top = high;
                            if (key == 0) sh.tops[wg][0] = high, sh.tops[wg][1] = near ? high : kApart;
                            sh.gain[par][gi][r] = __uint_as_float((uint32_t)(kGainBytes - top) << 23);
                            const float f = live ? ex2_approx(old - now) : 0.f;
                            sh.shrink[gi][r] = f;
                            sh.oshrink[gi][r] = f * __uint_as_float((uint32_t)(min(max(was - top, -126), 127) + 127) << 23);
                        }
                        named_bar_sync(bar, 128);
                        if (!fresh) {
                            const uint32_t shrink = shb + (uint32_t)offsetof(F, shrink) + (gi * RP + col0) * 4;
                            const uint32_t oshrink = shb + (uint32_t)offsetof(F, oshrink) + (gi * RP + col0) * 4;
                            const uint32_t ot = lanes + NS * RP + (kStream ? par * 2 + gi : par) * L::kO + col0;
#pragma unroll
                            for (int j = 0; j < NC; j += 4) {
                                const float4 f = lds4(shrink + j * 4);
                                l[j / 2] = mul2(l[j / 2], F2(f.x, f.y));
                                l[j / 2 + 1] = mul2(l[j / 2 + 1], F2(f.z, f.w));
                            }
#pragma unroll 1
                            for (int j = 0; j < kParts * NC; j += 8) {      // NC rows of each part
                                if (j % NC >= rows) continue;
                                const uint32_t at = ot + j / NC * RP + j % NC;
                                float o[8];
                                tmem_ld8_async(at, o);
                                const float4 f = lds4(oshrink + j % NC * 4), g = lds4(oshrink + j % NC * 4 + 16);
                                tmem_wait_ld();
                                o[0] *= f.x, o[1] *= f.y, o[2] *= f.z, o[3] *= f.w;
                                o[4] *= g.x, o[5] *= g.y, o[6] *= g.z, o[7] *= g.w;
                                tmem_st8(at, o);
                            }
                            tmem_wait_st();
                        }
                        most = sh.tops[wg][0];
                        shared = sh.tops[wg][1];
                    }
                    // Scores less their references: rounded products, as a reference is, so that a
                    // reference and the score that it comes from cancel whatever their size (a fused
                    // product of a score past 2^24 differs from it by powers of two, past 2^31 by more
                    // than a weight can hold).
#pragma unroll
                    for (int j = 0; j < NC; j += 4) {
                        const float4 m = lds4(mine + j * 4), f = lds4(qmul + j * 4);
                        add2(mul2(mul2(F2(x[j], x[j + 1]), km2), F2(f.x, f.y)), F2(m.x, m.y)).get(x[j], x[j + 1]);
                        add2(mul2(mul2(F2(x[j + 2], x[j + 3]), km2), F2(f.z, f.w)), F2(m.z, m.w)).get(x[j + 2], x[j + 3]);
                    }
                    if (masked && __any_sync(0xffffffffu, hidden > 0)) {        // -inf where a row does not see the key
#pragma unroll
                        for (int j = 0; j < NC; ++j)
                            if (j < hidden) x[j] = -INFINITY;
                    }
                    // This P^T buffer's last product is done.  (Of one team: the chunk before the
                    // last one's, which has been waited for above; of two, the team's last.)
                    if (kStream) wait(BAR(p_empty, b), use ^ 1, dead);
                    uint32_t top = 0;           // the largest halves
                    static_assert(NC == 16, "a thread's rows are one 16-byte piece of each part");
                    uint32_t c1[4], c2[4], c3[4], halves[NC / 2];
#pragma unroll
                    for (int j = 0; j < NC; ++j) x[j] = ex2_approx(x[j]);
                    // weight times gain times value scale (a weight of zero stays zero)
                    if (vb - shared <= kMostBytes) {
                        const float vm = __uint_as_float((uint32_t)max(vb - shared + kGainBytes - 127, 0) << 23);
#pragma unroll
                        for (int j = 0; j < NC; j += 2) halves[j / 2] = cvt_f16x2(mul2(F2(x[j], x[j + 1]), F2(vm, vm)));
                    } else {
                        const float vm = scale_of(vb);
#pragma unroll
                        for (int j = 0; j < NC; j += 4) {
                            const float4 g = lds4(gains + j * 4);
                            halves[j / 2] = cvt_f16x2(mul2(mul2(F2(x[j], x[j + 1]), F2(g.x, g.y)), F2(vm, vm)));
                            halves[j / 2 + 1] = cvt_f16x2(mul2(mul2(F2(x[j + 2], x[j + 3]), F2(g.z, g.w)), F2(vm, vm)));
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t h[2], t1[2], t2[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            h[k] = halves[2 * e + k];
                            top = max_f16x2(top, h[k]);
                            t1[k] = (h[k] + 0x00800080u) & 0xFF00FF00u;                     // rounded to e5m2
                            h[k] = mul_f16x2(sub_f16x2(h[k], t1[k]), kHalves2);
                            t2[k] = (h[k] + 0x00800080u) & 0xFF00FF00u;
                            h[k] = mul_f16x2(sub_f16x2(h[k], t2[k]), kHalves3) + 0x00800080u;   // the last part's upper bytes, rounded
                        }
                        c1[e] = upper_bytes(t1[0], t1[1]);
                        c2[e] = upper_bytes(t2[0], t2[1]);
                        c3[e] = upper_bytes(h[0], h[1]);
                    }
                    const uint32_t to = weights + b * kParts * L::kP;
                    sts4(to, c1[0], c1[1], c1[2], c1[3]);
                    sts4(to + L::kP, c2[0], c2[1], c2[2], c2[3]);
                    sts4(to + 2 * L::kP, c3[0], c3[1], c3[2], c3[3]);
                    if (masked && wg % kTeam == active - 1) {
                        // Values of positions that some row does not see: behind the
                        // length they become zero (a weight of zero does not silence a
                        // NaN), between the rows' last positions NaN do, and are added at
                        // the end to the rows that see them.
                        // (The slot's last V has been consumed: its product came before this P^T buffer's last.)
                        wait(BAR(v_full, i % NV), (i / NV) & 1, dead);
                        uint8_t* const tile = vslots + i % NV * L::kSlot;
                        if (kp >= w.len) {          // a thread's own row; lanes start at different banks
#pragma unroll
                            for (int e = 0; e < HD / 16; ++e)
                                *reinterpret_cast<uint4*>(tile + key * HD + (((e + lane) & (HD / 16 - 1)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                        }
                        const int from = max(0, last0 + 1 - (kp - key)), to = min(kChunk, w.len - (kp - key));
#pragma unroll 1
                        for (int t = from * (HD / 16) + key; t < to * (HD / 16); t += 128) {
                            uint4* const at = reinterpret_cast<uint4*>(tile + t * 16);
                            uint4 x = *at;
                            uint32_t* y = &x.x;
                            bool hit = false;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t n = ((y[k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;    // the bytes that are NaN
                                if (n) hit = true, y[k] &= ~((n >> 7) * 255u);
                            }
                            if (hit) {
                                *at = x;
                                sh.poison[par] = seg + 1;
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    tc_fence_before();
                    // Weights whose first part overflows (from 61440 on): the references move, and the chunk is taken again.
                    bool over = ((top + 0x04800480u) & 0x80008000u) != 0;
                    if (vb < most - kFarScale) {        // (no value, or one that is nothing beside the others)
                        float largest = 0.f;
#pragma unroll
                        for (int j = 0; j < NC; ++j) largest = fmaxf(largest, x[j]);
                        over = over || largest > kFarWeight;
                    }
                    if (!bar_any(bar, 128, over && !move) || move) break;
                }
#pragma unroll
                for (int j = 0; j < NC; j += 2) l[j / 2] = add2(l[j / 2], F2(x[j], x[j + 1]));
                fresh = false;
                arrive_if(BAR(s_empty, i % NS), speaks);
                arrive_if(BAR(c_empty, i % kScaleSlots), speaks);
                arrive_if(BAR(p_full, b), speaks);
            }
            unit += w.units;
            // sums over the warp's keys: lanes exchange halves until lane r holds row r, then
            // lanes of the same row are added
            if (rows > 0) {
                float v[NC];
#pragma unroll
                for (int e = 0; e < NC; e += 2) l[e / 2].get(v[e], v[e + 1]);
#pragma unroll
                for (int h = NC / 2; h >= 1; h >>= 1) {
                    const bool up = lane & h;
#pragma unroll
                    for (int e = 0; e < h; ++e) {
                        const float give = up ? v[e] : v[e + h], keep = up ? v[e + h] : v[e];
                        v[e] = keep + __shfl_xor_sync(0xffffffffu, give, h);
                    }
                }
                v[0] += __shfl_xor_sync(0xffffffffu, v[0], 16);
                if (lane < NC) sh.xl[par][gi][qd][col0 + lane] = v[0];
            }
            __syncwarp();
            arrive_if(BAR(l_full, par), lane == 0);
        }
    } else {
        // ---------------- the next segment's queries, and results: thread = head dimension ----------------
        regs_down<L::kResultRegs>();
        const int qd = warp & 3, d = qd * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(qd * 32) << 16);
        constexpr int kRowThreads = HD / 8, kPass = 128 / kRowThreads;     // 8 elements a thread; rows that the warpgroup splits at once
        constexpr int kAhead = RP / kPass < 4 ? RP / kPass : 4;            // and how many times that much is in flight
        const int b = d & (kRowThreads - 1), qrow = d / kRowThreads;
        Ring<2> qr;
        uint4 ahead[kAhead];
        auto fetch = [&](const Seg& s, int r0) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int r = r0 + k * kPass + qrow;
                if (r >= s.R) continue;
                const int t = token(s, r);
                ahead[k] = *reinterpret_cast<const uint4*>(p.q + (long long)(s.row0 + t) * p.q_stride +
                                                           (long long)(s.head * p.group + s.skip + r - t * p.group) * HD + b * 8);
            }
        };
        // Queries in two e4m3 parts with a power of two for each row.
        auto split_queries = [&](const Seg s, int par) {
            wait(BAR(q_empty, qr.at), qr.round ^ 1, dead);
            uint8_t* const tile = qs + qr.at * L::kQ;
#pragma unroll 1
            for (int r = qrow, k = 0; r - qrow < s.R; r += kPass) {
                if (k == 0) fetch(s, r - qrow);
                if (++k == kAhead) k = 0;
                const uint4 x = ahead[0];
#pragma unroll
                for (int e = 0; e + 1 < kAhead; ++e) ahead[e] = ahead[e + 1];
                const uint32_t* y = &x.x;
                uint32_t top = 0;               // largest finite magnitude
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t lo = y[k] & 0x7FFFu, hi = (y[k] >> 16) & 0x7FFFu;
                    if (lo < 0x7F80u) top = max(top, lo);
                    if (hi < 0x7F80u) top = max(top, hi);
                }
#pragma unroll
                for (int m = 1; m < kRowThreads; m <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
                const uint32_t f = max(top >> 7, 8u);           // its exponent: the row times 2^(134 - f) lies below 256
                const float mul = __uint_as_float((261u - f) << 23);
                uint32_t c1[4], c2[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float u = __uint_as_float(y[k] << 16), v = __uint_as_float(y[k] & 0xFFFF0000u);
                    u = isinf(u) ? __uint_as_float(0x7FC00000u) : u * mul;
                    v = isinf(v) ? __uint_as_float(0x7FC00000u) : v * mul;
                    c1[k] = split_e4m3(u, v);
                    c2[k] = split_e4m3(u, v);
                }
                if (r < s.R) {
                    uint8_t* at = tile + swizzled<HD>(r, b * 8);
                    *reinterpret_cast<uint2*>(at) = make_uint2(c1[0] | c1[1] << 16, c1[2] | c1[3] << 16);
                    *reinterpret_cast<uint2*>(at + L::kQPart) = make_uint2(c2[0] | c2[1] << 16, c2[2] | c2[3] << 16);
                    if (b == 0) sh.qmul[par][r] = __uint_as_float((f - 7u) << 23) * p.scale_log2;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            arrive_if(BAR(q_full, qr.at), lane == 0);
            arrive_if(BAR(r_full, par), lane == 0);
            qr.step();
        };
        int i = 0;                              // the segment's first unit
#pragma unroll 1
        for (int seg = -1;; ++seg) {            // the next segment's queries, then this one's results
            wait(BAR(seg_full, sr.at), sr.round, dead, plan8::wait_rounds(before));
            __syncwarp();
            if (bar_any(kResultBar, 128, raised(dead))) break;
            before = sh.segs[sr.at].units;
            const bool more = before != 0;
            if (more) split_queries(sh.segs[sr.at], (seg + 1) & 1);
            const int here = (sr.at + kSegs - 1) % kSegs;
            sr.step();
            if (seg < 0) {
                if (!more) break;
                continue;
            }
            const Seg w = sh.segs[here];
            const int par = seg & 1, last0 = w.last0;
            const int ga = kStream ? i & 1 : 0; // the team of the first unit; the other has none in a segment of one
            const bool two = kStream && w.units > 1, whole = w.slot < 0;
            i += w.units;
            if (qd == 0) wait(BAR(l_full, par), (seg >> 1) & 1, dead, plan8::wait_rounds(w.units));
            named_bar_sync(kResultBar, 128);
            if (d < w.R) {
                const int r = d;
                auto sum = [&](int g) { return sh.xl[par][g][0][r] + sh.xl[par][g][1][r] + sh.xl[par][g][2][r] + sh.xl[par][g][3][r]; };
                float ma = -sh.nref[par][ga][r], la = sum(ga);
                float fa = 1.f, fb = 0.f;
                if (two) {
                    const int gb = ga ^ (kGroups - 1);
                    const float mb = -sh.nref[par][gb][r], lb = sum(gb);
                    const float m = fmaxf(ma, mb);
                    fa = ex2_approx(ma - m);
                    fb = ex2_approx(mb - m);
                    la = la * fa + lb * fb;
                    ma = m;
                }
                const int t = token(w, r);
                if (whole) {                    // (a row without a position: zeros)
                    const float inv = last0 + t < 0 ? 0.f : rcp_approx(la);
                    fa *= inv;
                    fb *= inv;
                } else {
                    p.part_ml[(size_t)w.slot * RP + r] = make_float2(ma, la);
                }
                // the gain in O^T, a power of two, taken back
                auto undo = [&](int g) { return __uint_as_float((254u << 23) - __float_as_uint(sh.gain[par][g][r])); };
                fa *= undo(ga);
                if (two) fb *= undo(ga ^ (kGroups - 1));
                sh.row[par][r] = {{fa, fb}, t * p.out_stride + (long long)(r - t * p.group) * HD};
            }
            if (qd == 0) wait(BAR(o_full, par), (seg >> 1) & 1, dead);
            named_bar_sync(kResultBar, 128);
            const bool bad = sh.poison[par] == seg + 1;
            tc_fence_after();
            uint16_t* const out = p.out + (long long)w.row0 * p.out_stride + ((long long)w.head * p.group + w.skip) * HD + d;
            float* const part = p.part_o + (size_t)(whole ? 0 : w.slot) * RP * HD + d;
#pragma unroll 1
            for (int j0 = 0; j0 < w.R; j0 += 8) {
                // 8 rows' O^T of the first team (its three parts), and of the other
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll 1
                for (int g = 0; g < (two ? 2 : 1); ++g) {
                    const uint32_t at = lanes + NS * RP + (kStream ? par * 2 + (ga ^ g) : par) * L::kO + j0;
                    float x[8], u[8], v[8];
                    tmem_ld8_async(at, x);
                    tmem_ld8_async(at + RP, u);
                    tmem_ld8_async(at + 2 * RP, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        o[e] += (x[e] + (u[e] + v[e] * (1.f / kPart3)) * (1.f / kPart2)) * sh.row[par][j0 + e].f[g];
                }
                if (d < HD) {
                    if (bad)                    // of the positions that some row of the block sees and some does not
#pragma unroll 1
                        for (int t = max(last0 + 1, w.c0 * kChunk); t < min(last0 + token(w, w.R - 1) + 1, (w.c0 + w.units) * kChunk); ++t) {
                            const int page = p.tables[(size_t)w.q * p.table_pages + t / SPEC_PAGE];
                            if (page < 0 || page >= p.num_pages) continue;
                            const int code = p.vpool[(((size_t)page * p.hkv + w.head) * SPEC_PAGE + t % SPEC_PAGE) * HD + d];
                            if ((code & 0x7F) == 0x7F)
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    if (t <= last0 + token(w, j0 + e)) o[e] = __uint_as_float(0x7FC00000u);
                        }
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (j0 + e < w.R) out[sh.row[par][j0 + e].at] = f2bf(o[e]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (j0 + e < w.R) part[(j0 + e) * HD] = o[e];
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            arrive_if(BAR(o_empty, par), lane == 0);
            arrive_if(BAR(l_empty, par), lane == 0);
            arrive_if(BAR(seg_empty, here), lane == 0);
            if (!more) break;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && sh.dead && p.err) atomicCAS(p.err, 0, SPEC_PAGED_TIMEOUT);
    if (warp == kScoreWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kCols);
    }
#undef BAR
}

spec_status bad8(const char* what) {
    static thread_local char msg[192];
    snprintf(msg, sizeof msg, "spec_paged_attention_fp8: %s", what);
    return bad(msg);
}

// What the head layout has to satisfy; null when it does.
const char* head_error8(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t max_new) {
    if (head_dim != 64 && head_dim != 128) return "head_dim must be 64 or 128";
    if (n_kv_heads < 1 || n_kv_heads > 1024 || n_heads < n_kv_heads || n_heads % n_kv_heads)
        return "n_heads must be a multiple of n_kv_heads, 1..1024";
    if (n_heads / n_kv_heads > 128) return "at most 128 query heads per kv head";
    if (max_new < 1) return "max_new must be at least 1";
    return nullptr;
}

// Codes [d2][SPEC_PAGE][hd], read a page and head at a time, a row as wide as the swizzle.
bool encode8(CUtensorMap* map, const void* p, uint64_t hd, uint64_t d2) {
    const cuuint64_t dims[3] = {hd, SPEC_PAGE, d2}, strides[2] = {hd, hd * SPEC_PAGE};
    const cuuint32_t box[3] = {(cuuint32_t)hd, SPEC_PAGE, 1}, step[3] = {1, 1, 1};
    return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(p), dims, strides, box, step,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, hd == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD, int RP>
cudaError_t run8(Paged8Params& p, int ctas, cudaStream_t s) {
    const void* fn = (const void*)paged_attn8_kernel<HD, RP>;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Plan<HD, RP>::kBytes);
    if (e != cudaSuccess) return e;
    void* args[] = {&p};
    if ((e = launch(fn, dim3((unsigned)ctas), 32 * Plan<HD, RP>::kWarps, Plan<HD, RP>::kBytes, s, args)) != cudaSuccess || p.whole) return e;
    int rp = RP;
    void* jargs[] = {static_cast<PagedCommon*>(&p), &rp};
    return launch((const void*)paged_join_kernel<HD>, dim3((unsigned)ctas, 2 * (RP <= 16 ? 1 : RP / 16)), 32 * kJoinWarps, 0, s, jargs);
}

}  // namespace
}  // namespace sv

extern "C" {

using namespace sv;

spec_status spec_paged_attention_fp8_workspace(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t max_new,
                                               int32_t table_pages, size_t* out_bytes) {
    if (!out_bytes) return bad8("null pointer");
    if (const char* e = head_error8(n_heads, n_kv_heads, head_dim, max_new)) return bad8(e);
    if (table_pages < 1 || table_pages > SPEC_MAX_TABLE) return bad8("table_pages must be in 1..1048576");
    if (split::whole_pairs(table_pages)) {
        *out_bytes = 0;
        return SPEC_OK;
    }
    const int sms = current_sms();
    if (!sms) {
        set_last_error("spec_paged_attention_fp8_workspace: no current CUDA device");
        return SPEC_ERR_CUDA;
    }
    *out_bytes = Work(sms, split8::tile_height(n_heads / n_kv_heads, max_new), head_dim).bytes;
    return SPEC_OK;
}

spec_status spec_paged_attention_fp8(const void* d_q, int64_t q_stride, const int32_t* d_row_start, const int32_t* d_len,
                                     const int32_t* d_tables, int32_t table_pages, int32_t nseq, int32_t rows,
                                     int32_t max_new, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, float scale,
                                     const void* d_kpool, const void* d_vpool, const void* d_scales, int32_t num_pages,
                                     void* d_out, int64_t out_stride, int32_t* d_error_opt, void* d_work, size_t work_bytes,
                                     void* cuda_stream) {
    if (const char* e = head_error8(n_heads, n_kv_heads, head_dim, max_new)) return bad8(e);
    if (nseq < 0 || nseq > SPEC_MAX_SEQS) return bad8("nseq must be in 0..1024");
    if (rows < 0) return bad8("negative rows");
    if (table_pages < 1 || table_pages > SPEC_MAX_TABLE) return bad8("table_pages must be in 1..1048576");
    if (num_pages < 1 || num_pages > SPEC_MAX_PAGES) return bad8("num_pages must be in 1..33554431");
    if ((int64_t)num_pages * n_kv_heads > 0x7fffffff) return bad8("num_pages * n_kv_heads must fit int32");
    if (!(scale > 0.f) || !isfinite(scale)) return bad8("scale must be positive and finite");
    const int64_t row = (int64_t)n_heads * head_dim;
    if (q_stride < row || out_stride < row || (q_stride & 7) || (out_stride & 7) || q_stride >= (1ll << 38) ||
        out_stride >= (1ll << 38))
        return bad8("row strides must be multiples of 8, at least n_heads * head_dim and below 2^38");
    if (nseq == 0 || rows == 0) return SPEC_OK;
    const bool whole = split::whole_pairs(table_pages);
    if (!d_q || !d_row_start || !d_len || !d_tables || !d_kpool || !d_vpool || !d_scales || !d_out || (!whole && !d_work))
        return bad8("null pointer");
    if (misaligned(d_q, 16) || misaligned(d_out, 16) || misaligned(d_kpool, 16) || misaligned(d_vpool, 16) || misaligned(d_scales, 16))
        return bad8("queries, output, pools and scales must be 16-byte aligned");
    if (misaligned(d_row_start, 4) || misaligned(d_len, 4) || misaligned(d_tables, 4) || misaligned(d_error_opt, 4))
        return bad8("an int32 pointer is not 4-byte aligned");
    if (misaligned(d_work, 256)) return bad8("d_work is not 256-byte aligned");
    const int group = n_heads / n_kv_heads, rp = split8::tile_height(group, max_new), tile = split8::tile_rows(rp, group);
    // every unit has to fit int32, whatever the lengths on the device
    const int64_t pairs = ((int64_t)nseq + (int64_t)rows * group / tile) * n_kv_heads;
    if (pairs > 0x7fffffffll / ((table_pages + 1) / 2 + split8::kHead))
        return bad8("too much work for one call ((nseq + rows / tile) * n_kv_heads * table_pages / 2)");
    if (!whole && work_bytes < Work(1, rp, head_dim).bytes) return bad8("work_bytes is less than these heads need");
    const int sms = current_sms();
    if (!sms) {
        set_last_error("spec_paged_attention_fp8: no current CUDA device");
        return SPEC_ERR_CUDA;
    }
    const Work work(sms, rp, head_dim);
    if (!whole && work_bytes < work.bytes) return bad8("work_bytes is less than these heads need");
    if (!encode_fn()) {
        set_last_error("spec_paged_attention_fp8: the driver has no cuTensorMapEncodeTiled");
        return SPEC_ERR_CUDA;
    }
    Paged8Params p;
    if (!encode8(&p.mk, d_kpool, head_dim, (uint64_t)num_pages * n_kv_heads) ||
        !encode8(&p.mv, d_vpool, head_dim, (uint64_t)num_pages * n_kv_heads)) {
        set_last_error("spec_paged_attention_fp8: a tensor map could not be made");
        return SPEC_ERR_CUDA;
    }
    p.q = static_cast<const uint16_t*>(d_q);
    p.q_stride = q_stride;
    p.vpool = static_cast<const uint8_t*>(d_vpool);
    p.scales = static_cast<const uint8_t*>(d_scales);
    p.row_start = d_row_start;
    p.len = d_len;
    p.tables = d_tables;
    p.table_pages = table_pages;
    p.nseq = nseq;
    p.rows = rows;
    p.hkv = n_kv_heads;
    p.group = group;
    p.tokens = split8::tile_tokens(tile, group);
    p.tile = tile;
    p.whole = whole;
    p.scale_log2 = scale * 1.44269504088896340736f;
    p.num_pages = num_pages;
    p.out = static_cast<uint16_t*>(d_out);
    p.out_stride = out_stride;
    p.err = d_error_opt;
    uint8_t* wk = static_cast<uint8_t*>(d_work);
    p.part_o = reinterpret_cast<float*>(wk + work.o);
    p.part_ml = reinterpret_cast<float2*>(wk + work.ml);
    p.meta = reinterpret_cast<Meta*>(wk + work.meta);
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    cudaError_t e;
    if (head_dim == 128)
        e = rp == 16 ? run8<128, 16>(p, sms, s) : rp == 32 ? run8<128, 32>(p, sms, s) : run8<128, 64>(p, sms, s);
    else
        e = rp == 16 ? run8<64, 16>(p, sms, s) : rp == 32 ? run8<64, 32>(p, sms, s) : run8<64, 64>(p, sms, s);
    return e == cudaSuccess ? SPEC_OK : failed(e);
}

}  // extern "C"
