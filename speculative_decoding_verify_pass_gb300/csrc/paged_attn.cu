// Attention of each sequence's newest positions over a paged cache, on the
// fifth-generation tensor cores (tcgen05, accumulators in tensor memory).
//
// For a kv head, R = tokens * G query rows (G query heads per kv head) meet
// every key, so keys and head dimensions run along the 128 tensor-memory lanes
// and the rows are the narrow side.  Per 128-position chunk (two pages):
//     S^T = K Q^T      M = 128 keys,       N = R rounded up to 16, K = head dim
//     P^T = exp2(scale log2e S^T - m)
//     O^T += V^T P^T   M = head dimensions, N = as above,          K = 128 keys
// TMA tiles of 64 positions x 64 dimensions land with the 128-byte swizzle and
// are MMA operands as they lie: K rows are K-major, V rows are MN-major (V^T
// without a transpose).  P^T is kept as a bf16 high and a bf16 low part (about
// 16 significant bits), so that only the result's own rounding shows; up to 32
// rows the two parts lie side by side in one product's N (an MMA that narrow
// costs the same for 16 columns as for 64), with a column each in tensor memory.
//
// The softmax needs no maximum: m is a reference that a row takes from the score
// of one key, the first of its first chunk.  A score may exceed it by 40 in log2
// units (a weight of 2^40, which fp32 and bf16 hold), and only when one exceeds it
// by more do the row's reference, sum and O^T move to the chunk's maximum.  So per chunk and
// element there is one multiply-add, one exp2, one add to the thread's own
// partial sum and the two roundings; nothing crosses lanes until the segment
// ends.
//
// Roles, by warpgroup: 0 and 1 softmax (thread = key); 2 one warp each for the
// MMAs of S^T, the MMAs of O^T, the copies of V, and the list of segments with the
// copies of Q and K (K runs ahead of V: one copying warp would wait for a V slot
// with K slots free); 3 results (thread = head dimension).  Up to 64 rows the two
// softmax warpgroups take alternate chunks, each with its own reference, sum and
// O^T (joined with the results): a warp's chain of dependent instructions is what a
// chunk of few rows costs, and two chains run side by side.  128 rows are halved
// between the warpgroups instead (shared memory has no room for two P^T).  O^T and
// the sums are double buffered by segment, so that a segment's results are written
// while the next one runs.  One CTA per SM, each with the same number of chunks
// (paged_split.h); a second kernel joins the pairs that were split between CTAs.
//
// What bounds it, on a GB300 whose copies reach 6.8 TB/s (K and V of 8 heads of 128,
// GPU time): HBM for long caches and full batches (64 ragged decodes up to 8192
// positions 168 us, 6.7 TB/s; one sequence of 100003 positions 65.3 us, 6.3 TB/s, of
// which about 5 us are the launch, the first copies' latency, the results and the
// join); the chain through a chunk at 128 rows (100003 positions 85 us): of about 3050
// cycles at 1.93 GHz, against 2830 of HBM time, scores and the vote on references take
// 1200, weights and P^T 1080, the wait for the chunk before's product 280 (there is one
// P^T), for S^T 320; latency for short ones (one sequence
// of 128 positions 5.7 us, 300 6.9, 4104 with 8 rows 11.8: about 1 us each for the
// launch, the lengths, the page table, the first tile, the chain through the two
// products and, where pairs are split, 3 us for the join); work per segment, since
// CTAs share chunks evenly and not segments: at 128 rows each one more makes a CTA
// about 7000 cycles later (24 sequences of up to 8000: 75 us with one segment, 102
// with eight, cycle counters included), and instruction fetch for many short sequences
// of 64-wide heads (200 of up to 1500 positions with ragged blocks 39 us against 19.5
// of HBM time); hidden chunks for blocks longer than a tile (6000 rows of a prompt
// 1.5 ms against 0.15 of arithmetic).
#include "paged_core.cuh"
#include "paged_plan.h"

namespace sv {
namespace {

using plan::kFewSeqs;
using plan::kSegs;
using plan::kWarps;
using plan::Plan;
using plan::Seg;

constexpr float kWide = 1 << 24;        // size of a reference from which its own rounding counts
constexpr int kSoftWarps = 8, kScoreWarp = 8, kLoadVWarp = 10, kLoadKWarp = 11, kResultWarp = 12;
constexpr int kThreads = 32 * kWarps;
constexpr float kLimit = 40.f;          // log2 by which a score may exceed its row's reference
constexpr int kSoftBar = 1, kResultBar = 3; // named barriers: one per softmax warpgroup, the results' warpgroup

struct PagedParams : PagedCommon {
    CUtensorMap mq, mk, mv;
    const uint16_t* vpool;
};

__device__ __forceinline__ void tma3(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// Shared-memory matrix descriptor with the 128-byte swizzle.  K-major: 8-row
// groups sbo apart (lbo unused).  MN-major: 64-element column blocks lbo apart,
// 8-row (k) groups sbo apart.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}

// The upper half of such a descriptor (stride, version, swizzle).
constexpr uint32_t hi_sw128(uint32_t sbo) { return (sbo >> 4) | (1u << 14) | (2u << 29); }

// 32 consecutive fp32 columns of this warp's 32 lanes, not waited for.
__device__ __forceinline__ void tmem_ld32_async(uint32_t t, float* v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
          "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
          "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(t)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// Wait bounded in time (2^31 cycles, about a second, whatever one poll takes; more rounds
// of that while nothing else has given up); one that gives up raises `dead`.  Inline (a call
// would fix the registers that setmaxnreg moves) and short: the roles' loops share one
// instruction cache.
// A role whose wait failed waits no more.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* dead, int rounds = 1) {
    uint32_t t0 = cycles();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity))
        if (cycles() - t0 > 0x7fffffffu) {
            if (--rounds > 0 && !*dead) {
                t0 = cycles();
                continue;
            }
            *dead = 1;
            return false;
        }
    return true;
}
// After a failed wait: let what is in flight finish before the CTA ends.
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
    for (uint32_t i = 0; i < (1u << 20) && !mbar_try_wait(bar, parity); ++i) __nanosleep(64);
}

// D[tmem] (+)= A B^T with descriptors in halves: the upper one is a constant of the
// operand's layout, so that stepping along k is one 32-bit addition.
__device__ __forceinline__ void umma_lo(uint32_t d, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(accumulate)
        : "memory");
}

// A CTA's segments in order.
struct Walk {
    const PagedParams& p;
    const int* first;           // [nseq + 1] in shared memory
    const int *start, *lens;    // row starts and lengths: in shared memory when they are few
    int u, end;                 // next unit, end of the CTA's range
    int q = 0, q1 = 0;          // sequence, the end of its units
    int rows = 0, len = 0, row_base = 0, chunks = 1;
    // the segment
    int head = 0, block = 0, c0 = 0, c1 = 0, R = 0, seg = -1;

    __device__ Walk(const PagedParams& pp, const int* f, const int* s, const int* n, int begin, int e)
        : p(pp), first(f), start(s), lens(n), u(begin), end(e) {}
    __device__ __forceinline__ void sequence() {
        q1 = first[q + 1];
        row_base = start[q];
        rows = start[q + 1] - row_base;
        len = lens[q];
        chunks = split::chunks_of(len);
    }
    __device__ __forceinline__ bool next() {
        if (u >= end) return false;
        if (seg < 0) {                          // where the range begins
            q = split::sequence_of(first, p.nseq, u);
            sequence();
            const int at = u - first[q], pair = at / chunks;
            block = pair / p.hkv;
            head = pair - block * p.hkv;
            c0 = at - pair * chunks;
            if (p.whole && c0 > 0) {            // this pair begins in another CTA's range, which takes it
                u += chunks - c0;
                if (u >= end) return false;
                step();
            }
        } else {
            step();
        }
        c1 = p.whole ? chunks : min(chunks, c0 + end - u);
        R = min(p.tokens, rows - block * p.tokens) * p.group;
        u += c1 - c0;
        ++seg;
        return true;
    }
    // the pair after the current one
    __device__ __forceinline__ void step() {
        c0 = 0;
        if (u >= q1) {
            do ++q;
            while (first[q + 1] <= u);          // sequences without units
            sequence();
            block = head = 0;
        } else if (++head == p.hkv) {
            head = 0;
            ++block;
        }
    }
    __device__ __forceinline__ bool whole() const { return c0 == 0 && c1 == chunks; }
    // last position that the block's first token sees
    __device__ __forceinline__ int last0() const { return len - rows + block * p.tokens; }
    // the segment's pair, for the join
    __device__ Meta meta(const split::Deal& deal) const {
        const int pair_begin = u - c1, owner = deal.cta(pair_begin);
        Meta m;
        m.count = deal.parts(owner, pair_begin + chunks);
        m.owner = owner;
        m.slot = 2 * owner + (pair_begin == deal.begin(owner) ? 0 : 1);
        m.rows = R;
        m.head = head * p.group;
        m.row0 = row_base + block * p.tokens;
        m.last0 = last0();
        m.skip = 0;
        return m;
    }
};

template <int HD, int RP>
__global__ void __block_size__((kThreads, 1, 1)) __maxnreg__(128) paged_attn_kernel(const __grid_constant__ PagedParams p) {
    using L = Plan<HD, RP>;
    constexpr bool kStream = L::kStream, kStack = L::kStack;
    constexpr int NK = L::NK, NV = L::NV, NP = L::NP, NQ = L::NQ;
    constexpr int NC = kStream ? RP : RP / 2;   // rows of a softmax thread
    // rows that a softmax thread handles or skips together: more make longer runs of
    // independent instructions, fewer waste less on tiles that are not full
    constexpr int kSpan = NC <= 16 ? 8 : NC <= 32 ? 16 : 32;
    constexpr int kGroups = L::kGroups;
    constexpr int kArrive = kStream ? 4 : 8;    // warps that read an S^T and write a P^T
    constexpr int kReaders = kSoftWarps + 3 + 4;    // warps that read the list of segments
    constexpr int kPieces = L::kPieces, kPieceRows = kChunk / kPieces;
    extern __shared__ uint8_t smem_raw[];
    __shared__ plan::Fixed<RP> sh;
    auto& k_full = sh.k_full; auto& k_empty = sh.k_empty; auto& v_full = sh.v_full; auto& v_empty = sh.v_empty;
    auto& q_full = sh.q_full; auto& q_empty = sh.q_empty; auto& s_full = sh.s_full; auto& s_empty = sh.s_empty;
    auto& p_full = sh.p_full; auto& p_empty = sh.p_empty; auto& o_full = sh.o_full; auto& o_empty = sh.o_empty;
    auto& l_full = sh.l_full; auto& l_empty = sh.l_empty; auto& seg_full = sh.seg_full; auto& seg_empty = sh.seg_empty;
    auto& fin = sh.fin; auto& tmem_base = sh.tmem_base; auto& dead = sh.dead; auto& total = sh.total;
    auto& poison = sh.poison; auto& first = sh.first; auto& few_start = sh.few_start; auto& few_len = sh.few_len;
    auto& warp_sum = sh.warp_sum; auto& segs = sh.segs; auto& nref = sh.nref; auto& xl = sh.xl;
    auto& weight = sh.weight; auto& tok = sh.tok; auto& col_off = sh.col_off;

    uint8_t* base = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* kslots = base;
    uint8_t* vslots = kslots + NK * L::kSlot;
    uint8_t* qs = vslots + NV * L::kPiece + 1024;       // 1 KB: an M = 128 MMA over 64 dimensions reads past its slot
    uint8_t* ps = qs + NQ * L::kQ;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < NK; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < NQ; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], kArrive);
            mbar_init(&o_full[i], 1);
            mbar_init(&o_empty[i], 4);
            mbar_init(&l_full[i], kSoftWarps);
            mbar_init(&l_empty[i], 4);
            mbar_init(&fin[i], 1);
            poison[i] = 0;
        }
        for (int i = 0; i < NP; ++i) {
            mbar_init(&p_full[i], kArrive);
            mbar_init(&p_empty[i], 1);
        }
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(&seg_full[i], 1);
            mbar_init(&seg_empty[i], kReaders);
        }
        fence_barrier_init();
        dead = 0;
        first[0] = 0;
    }
#pragma unroll 1
    for (int i = tid; i < RP; i += kThreads) {
        const int t = i / p.group;
        tok[i] = t;
        col_off[i] = t * p.out_stride + (long long)(i - t * p.group) * HD;
    }
    if (warp == kScoreWarp) tmem_alloc(&tmem_base, L::kCols);
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
                    few_start[q] = r0;
                    few_start[q + 1] = r1;      // the next sequence's r0, the same word
                    few_len[q] = n;
                }
                if (bad_rows || bad_len) {
                    if (blockIdx.x == 0 && p.err) atomicCAS(p.err, 0, bad_rows ? SPEC_PAGED_BAD_ROWS : SPEC_PAGED_BAD_LENGTH);
                } else {
                    v[k] = split::units_of(r1 - r0, n, p.tokens, p.hkv);
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
            if (lane == 31) warp_sum[warp] = inc;
            __syncthreads();
#pragma unroll 1
            for (int w = 0; w < warp && w * 64 < p.nseq; ++w) run += warp_sum[w];
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            run += v[k];
            if (tid * 2 + k < p.nseq) first[tid * 2 + k + 1] = (int)run;
        }
        if (tid == (p.nseq - 1) / 2) {
            total = run > 0x7fffffff ? 0 : (int)run;
            if (run > 0x7fffffff && blockIdx.x == 0 && p.err) atomicCAS(p.err, 0, SPEC_PAGED_BAD_ROWS);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    const split::Deal deal(total, gridDim.x);
    const int begin = deal.begin(blockIdx.x), end = deal.begin(blockIdx.x + 1);
    volatile int* deadp = &dead;
    Ring<kSegs> sr;                             // every role's place in the list of segments
    auto take = [&](bool one) {                 // the next segment; `one`: this thread alone stands for its warp
        wait(&seg_full[sr.at], sr.round, deadp);
        const Seg s = segs[sr.at];
        if (!one) __syncwarp();
        if (one || lane == 0) mbar_arrive(&seg_empty[sr.at]);
        sr.step();
        return s;
    };

    if (warp >= kScoreWarp && warp < kResultWarp) {
        regs_down<L::kIssueRegs>();
        if (warp == kLoadKWarp) {
            // ---------------- the list of segments, Q and K copies, and what the join kernel has to do here ----------------
            const bool few = p.nseq <= kFewSeqs;
            Walk w(p, first, few ? few_start : p.row_start, few ? few_len : p.len, begin, end);
            Meta into = {}, from = {};
            Ring<NK> kr;
            Ring<NQ> qr;
            bool ok = true;
#pragma unroll 1
            for (bool more = true; more && ok;) {
                more = w.next();
                Seg s = {};                     // no units: the list ends
                if (more) {
                    s.c0 = w.c0;
                    s.units = w.c1 - w.c0;
                    s.R = w.R;
                    s.last0 = w.last0();
                    s.len = w.len;
                    s.q = w.q;
                    s.head = w.head;
                    s.row0 = w.row_base + w.block * p.tokens;
                    s.slot = w.whole() ? -1 : 2 * (int)blockIdx.x + (w.u - s.units == begin ? 0 : 1);
                }
                ok = __all_sync(0xffffffffu, wait(&seg_empty[sr.at], sr.round ^ 1, deadp));
                if (!ok) break;
                if (lane == 0) {
                    segs[sr.at] = s;
                    mbar_arrive(&seg_full[sr.at]);
                }
                sr.step();
                if (!more) break;
                ok = __all_sync(0xffffffffu, wait(&q_empty[qr.at], qr.round ^ 1, deadp));
                if (!ok) break;
                if (elect_one()) {
                    uint64_t* qf = &q_full[qr.at];
                    mbar_arrive_expect_tx(qf, (uint32_t)(p.tokens * p.group * HD * 2));
#pragma unroll
                    for (int hf = 0; hf < HD / 64; ++hf)
                        tma3(qs + qr.at * L::kQ + hf * RP * 128, &p.mq, hf * 64, s.head * p.group, s.row0, qf);
                }
                __syncwarp();
                qr.step();
                PageWalk pages;
#pragma unroll 1
                for (int k = 0; k < s.units; ++k) {
                    pages.at(p, s, k, lane);
                    ok = __all_sync(0xffffffffu, wait(&k_empty[kr.at], kr.round ^ 1, deadp));
                    if (!ok) break;
                    if (elect_one()) {
                        uint64_t* full = &k_full[kr.at];
                        uint8_t* dst = kslots + kr.at * L::kSlot;
                        mbar_arrive_expect_tx(full, (uint32_t)(pages.count * SPEC_PAGE * HD * 2));
#pragma unroll
                        for (int hf = 0; hf < HD / 64; ++hf) {
                            if (pages.count > 0) tma3(dst + hf * kChunk * 128, &p.mk, hf * 64, 0, pages.z0, full);
                            if (pages.count > 1) tma3(dst + hf * kChunk * 128 + SPEC_PAGE * 128, &p.mk, hf * 64, 0, pages.z1, full);
                        }
                    }
                    __syncwarp();
                    kr.step();
                }
                if (w.seg == 0 && w.c0 > 0) into = w.meta(deal);
            }
            if (lane == 0 && !p.whole) {
                if (w.seg >= 0 && w.c1 < w.chunks && w.u - w.c1 >= begin) from = w.meta(deal);
                p.meta[2 * blockIdx.x] = into;
                p.meta[2 * blockIdx.x + 1] = from;
            }
            if (lane == 0 && *deadp) {          // every buffer's last copy, as far as one was issued
#pragma unroll 1
                for (int i = 0; i < NK; ++i) drain(&k_full[i], i < kr.at ? kr.round : kr.round ^ 1);
#pragma unroll 1
                for (int i = 0; i < NQ; ++i) drain(&q_full[i], i < qr.at ? qr.round : qr.round ^ 1);
            }
        } else if (warp == kLoadVWarp) {
            // ---------------- V copies ----------------
            Ring<NV> vr;
            bool ok = true;
#pragma unroll 1
            for (;;) {
                const Seg s = take(false);
                ok = __all_sync(0xffffffffu, !*deadp);
                if (!ok || s.units == 0) break;
                PageWalk pages;
#pragma unroll 1
                for (int k = 0; k < s.units && ok; ++k) {
                    pages.at(p, s, k, lane);
#pragma unroll 1
                    for (int v = 0; v < L::kPieces; ++v) {
                        ok = __all_sync(0xffffffffu, wait(&v_empty[vr.at], vr.round ^ 1, deadp));
                        if (!ok) break;
                        const int count = kPieces == 1 ? pages.count : pages.count > v ? 1 : 0;
                        if (elect_one()) {
                            uint64_t* full = &v_full[vr.at];
                            uint8_t* dst = vslots + vr.at * L::kPiece;
                            mbar_arrive_expect_tx(full, (uint32_t)(count * SPEC_PAGE * HD * 2));
#pragma unroll
                            for (int hf = 0; hf < HD / 64; ++hf) {
                                if (count > 0) tma3(dst + hf * kPieceRows * 128, &p.mv, hf * 64, 0, v ? pages.z1 : pages.z0, full);
                                if (count > 1) tma3(dst + hf * kPieceRows * 128 + SPEC_PAGE * 128, &p.mv, hf * 64, 0, pages.z1, full);
                            }
                        }
                        __syncwarp();
                        vr.step();
                    }
                }
                if (!ok) break;
            }
            if (lane == 0 && *deadp) {
#pragma unroll 1
                for (int i = 0; i < NV; ++i) drain(&v_full[i], i < vr.at ? vr.round : vr.round ^ 1);
            }
        } else if (warp == kScoreWarp) {
            // ---------------- MMAs of S^T (one elected thread) ----------------
            if (elect_one()) {
                Ring<NK> ks;
                Ring<NQ> qr;
                Ring<2> sb;
                const uint32_t sa = smem_u32(kslots), qa = smem_u32(qs);
                bool ok = true;
#pragma unroll 1
                while (ok) {
                    const Seg s = take(true);
                    ok = !*deadp;
                    if (!ok || s.units == 0) break;
                    ok = wait(&q_full[qr.at], qr.round, deadp);
                    const uint32_t id = umma_idesc_bf16(128, (s.R + 15) & ~15);
                    const uint32_t dq = (uint32_t)desc_sw128(qa + qr.at * L::kQ, 16, 1024);
                    constexpr uint32_t kHi = hi_sw128(1024);
#pragma unroll 1
                    for (int k = 0; k < s.units && ok; ++k) {
                        ok = wait(&k_full[ks.at], ks.round, deadp) && wait(&s_empty[sb.at], sb.round ^ 1, deadp);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t dk = (uint32_t)desc_sw128(sa + ks.at * L::kSlot, 16, 1024);
#pragma unroll
                        for (int e = 0; e < HD / 16; ++e)
                            umma_lo(tmem + sb.at * RP, dk + (e >> 2) * (kChunk * 128 >> 4) + (e & 3) * 2, kHi,
                                    dq + (e >> 2) * (RP * 128 >> 4) + (e & 3) * 2, kHi, id, e > 0);
                        umma_commit(&s_full[sb.at]);
                        umma_commit(&k_empty[ks.at]);
                        ks.step();
                        sb.step();
                    }
                    if (ok) umma_commit(&q_empty[qr.at]);
                    qr.step();
                }
                if (!ok || *deadp) {
                    umma_commit(&fin[0]);
                    drain(&fin[0], 0);
                }
            }
        } else {   // warp 9
            // ---------------- MMAs of O^T (one elected thread) ----------------
            if (elect_one()) {
                Ring<NV> vs;
                Ring<NP> pr;
                const uint32_t sa = smem_u32(vslots), pa = smem_u32(ps);
                bool ok = true;
                int j = 0;                      // unit
#pragma unroll 1
                for (int seg = 0; ok; ++seg) {
                    const Seg s = take(true);
                    ok = !*deadp;
                    if (!ok || s.units == 0) break;
                    ok = wait(&o_empty[seg & 1], ((seg >> 1) & 1) ^ 1, deadp);
                    // A = V^T and B = P^T, both MN-major
                    const uint32_t id = umma_idesc_bf16(128, kStack ? 2 * RP : (s.R + 15) & ~15) | (1u << 15) | (1u << 16);
#pragma unroll 1
                    for (int k = 0; k < s.units && ok; ++k, ++j) {
                        ok = wait(&p_full[pr.at], pr.round, deadp);
                        const uint32_t dp = (uint32_t)umma_desc_kmajor(pa + pr.at * 2 * L::kP, 128, kChunk * 16);
                        constexpr uint32_t kHiV = hi_sw128(1024), kHiP = (kChunk * 16 >> 4) | (1u << 14);
                        const int og = kStream ? (seg & 1) * 2 + (j & 1) : seg & 1;
                        const uint32_t o = tmem + 2 * RP + og * L::kO;
                        const bool more = k >= kGroups;     // this O^T holds earlier chunks
#pragma unroll
                        for (int v = 0; v < kPieces; ++v) {
                            ok = ok && wait(&v_full[vs.at], vs.round, deadp);
                            if (!ok) break;
                            tc_fence_after();
                            const uint32_t dv = (uint32_t)desc_sw128(sa + vs.at * L::kPiece, HD == 128 ? kPieceRows * 128 : 1024, 1024);
#pragma unroll
                            for (int part = 0; part < (kStack ? 1 : 2); ++part)
#pragma unroll
                                for (int e = 0; e < kPieceRows / 16; ++e)
                                    umma_lo(o, dv + e * (2048 >> 4), kHiV,
                                            dp + part * (L::kP >> 4) + (v * (kPieceRows / 16) + e) * (256 >> 4), kHiP, id,
                                            more || (v | part | e) != 0);
                            umma_commit(&v_empty[vs.at]);
                            vs.step();
                        }
                        if (!ok) break;
                        umma_commit(&p_empty[pr.at]);
                        pr.step();
                    }
                    if (ok) umma_commit(&o_full[seg & 1]);
                }
                if (!ok || *deadp) {
                    umma_commit(&fin[1]);
                    drain(&fin[1], 0);
                }
            }
        }
        __syncwarp();
    } else if (warp < kSoftWarps) {
        // ---------------- softmax: thread = key ----------------
        regs_up<L::kSoftRegs>();
        const int wg = warp >> 2, qd = warp & 3;
        const uint32_t lanes = tmem + ((uint32_t)(qd * 32) << 16);
        const int key = qd * 32 + lane;
        const int col0 = kStream ? 0 : wg * NC; // the thread's first row
        const int gi = kStream ? wg : 0;        // its reference and O^T
        const int bar = kSoftBar + wg;
        int i = 0;                              // unit
        Ring<NV> vs;                            // slot of the next unit's V
        bool ok = true;
#pragma unroll 1
        for (int seg = 0;; ++seg) {
            const Seg w = take(false);
            if (bar_any(bar, 128, *deadp != 0) || w.units == 0) break;   // after a wait that gave up, all of the warpgroup leaves
            const int par = seg & 1, last0 = w.last0, rows = w.R - col0;   // live rows of this thread
            float* const mine = nref[par][gi];
            ok = ok && wait(&l_empty[par], ((seg >> 1) & 1) ^ 1, deadp);   // the results of two segments ago have been read
            F2 l[NC / 2];
#pragma unroll
            for (int j = 0; j < NC / 2; ++j) l[j] = F2(0.f, 0.f);
            bool fresh = true, wide = false;   // wide: a reference past 2^24, every chunk takes its scores again
#pragma unroll 1
            for (int c = w.c0; c < w.c0 + w.units; ++c, ++i) {
                const Ring<NV> v0 = vs;         // the slots of the chunk's V: its first page's,
                if (kPieces == 2) vs.step();
                const Ring<NV> v1 = vs;         // and its second's
                vs.step();
                if (kStream && (i & 1) != wg) continue;
                const uint32_t st = lanes + (i & 1) * RP + col0;
                const int kp = c * kChunk + key;
                const bool masked = (c + 1) * kChunk - 1 > last0;   // some row does not see all of the chunk
                ok = ok && wait(&s_full[i & 1], (i >> 1) & 1, deadp);
                tc_fence_after();
                float s[NC];
                // this thread's P^T buffer is free (and its rows' O^T complete) once their last product is
                auto product_done = [&]() {
                    ok = ok && wait(&p_empty[kStream ? i & 1 : 0], ((kStream ? i >> 1 : i) & 1) ^ 1, deadp);
                };
#pragma unroll 1
                for (bool moved = false;; moved = true) {
                    // the chunk's scores, -inf where a row does not see the key
#pragma unroll
                    for (int j = 0; j < NC; j += kSpan)
                        if (j < rows) {
                            if constexpr (kSpan == 8) tmem_ld8_async(st + j, s + j);
                            else if constexpr (kSpan == 16) tmem_ld16_async(st + j, s + j);
                            else tmem_ld32_async(st + j, s + j);
                        }
                    tmem_wait_ld();
                    if (masked) {
                        // rows are in token order: the key is hidden from the tokens before it
                        const int hidden = min(max(kp - last0, 0), RP) * p.group - col0;
#pragma unroll
                        for (int j = 0; j < NC; ++j)
                            if (j < hidden) s[j] = -INFINITY;
                    }
                    if (rows <= 0) break;
                    bool big = wide;
                    if (fresh) {                // references: the scores of the chunk's first key
                        if (key == 0) {
#pragma unroll
                            for (int j = 0; j < NC; j += 4)
                                *reinterpret_cast<float4*>(&mine[col0 + j]) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
                        }
                        named_bar_sync(bar, 128);
                        if (key < NC) {
                            const float m = mine[col0 + key] * p.scale_log2;
                            mine[col0 + key] = key >= rows ? -INFINITY : m > kNone ? -m : -kNone;   // rows past R weigh nothing
                            big = fabsf(m) > kWide && m > kNone && key < rows;
                        }
                        named_bar_sync(bar, 128);
                    }
                    const float k = moved ? 1.f : p.scale_log2;
                    const F2 k2(k, k);
                    float top[2] = {kNone, kNone};
#pragma unroll
                    for (int j0 = 0; j0 < NC; j0 += kSpan)
                        if (j0 < rows) {
#pragma unroll
                            for (int j = j0; j < j0 + kSpan; j += 4) {
                                const float4 m = *reinterpret_cast<const float4*>(&mine[col0 + j]);
                                fma2(F2(s[j], s[j + 1]), k2, F2(m.x, m.y)).get(s[j], s[j + 1]);
                                fma2(F2(s[j + 2], s[j + 3]), k2, F2(m.z, m.w)).get(s[j + 2], s[j + 3]);
                                top[j / 4 & 1] = fmaxf(top[j / 4 & 1], fmaxf(fmaxf(s[j], s[j + 1]), fmaxf(s[j + 2], s[j + 3])));
                            }
                        }
                    if (moved || !bar_any(bar, 128, big || fmaxf(top[0], top[1]) > kLimit)) break;
                    // The references move up to the chunk's maxima, the sums and O^T
                    // with them, and the scores are taken again.  So that a reference and the
                    // score that it comes from cancel whatever their size, the scores are then
                    // rounded products, as it is: the fused product of a score past 2^24 differs
                    // from it by powers of two, past 2^31 by more than a weight can hold.
                    product_done();
                    tc_fence_after();
                    float (*const mx)[RP] = xl[par][gi];
#pragma unroll 1
                    for (int j = 0; j < NC && j < rows; j += 8) {
                        float x[8];
                        tmem_ld8_async(st + j, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] *= p.scale_log2;
                        tmem_st8(st + j, x);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float m = warp_max_exact(kp > last0 + tok[col0 + j + e] ? -INFINITY : x[e]);
                            if (lane == 0) mx[qd][col0 + j + e] = m;
                        }
                    }
                    named_bar_sync(bar, 128);
                    tmem_wait_st();
                    float now = 0.f;
                    if (key < NC) {             // one thread per row: the new reference, and what the old weights shrink by
                        const int r = col0 + key;
                        const float m = fmaxf(fmaxf(mx[0][r], mx[1][r]), fmaxf(mx[2][r], mx[3][r]));
                        const float old = -mine[r];
                        now = key < rows ? fmaxf(old, m) : INFINITY;
                        mine[r] = -now;
                        mx[0][r] = key < rows ? ex2_approx(old - now) : 0.f;
                    }
                    wide = bar_any(bar, 128, key < rows && fabsf(now) > kWide && now > kNone);
#pragma unroll
                    for (int j = 0; j < NC; j += 2) {
                        float x, y;
                        l[j / 2].get(x, y);
                        l[j / 2] = F2(x * mx[0][col0 + j], y * mx[0][col0 + j + 1]);
                    }
                    if (!fresh) {
                        const uint32_t ot = lanes + 2 * RP + (kStream ? par * 2 + wg : par) * L::kO + col0;
#pragma unroll 1
                        for (int j = 0; j < (kStack ? 2 * NC : NC); j += 8)   // stacked: the low part's columns follow
                            if ((kStack ? j & (NC - 1) : j) < rows) {
                                float o[8];
                                tmem_ld8_async(ot + j, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 8; ++e) o[e] *= mx[0][col0 + (j & (NC - 1)) + e];
                                tmem_st8(ot + j, o);
                            }
                        tmem_wait_st();
                    }
                    fresh = false;
                    named_bar_sync(bar, 128);   // everyone has read mx
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_empty[i & 1]);
                fresh = false;
                product_done();
                uint8_t* ph = ps + (kStream ? i & 1 : 0) * 2 * L::kP + (col0 >> 3) * (kChunk * 16) + key * 16;
#pragma unroll
                for (int j0 = 0; j0 < NC; j0 += kSpan)
                    if (j0 < rows) {
#pragma unroll
                        for (int j = j0; j < j0 + kSpan; j += 8) {
                            uint32_t hi[4], lo[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const F2 x(ex2_approx(s[j + 2 * e]), ex2_approx(s[j + 2 * e + 1]));
                                l[j / 2 + e] = add2(l[j / 2 + e], x);
                                float a, b;
                                x.get(a, b);
                                hi[e] = cvt_bf16x2(a, b);
                                const F2 h(__uint_as_float(hi[e] << 16), __uint_as_float(hi[e] & 0xFFFF0000u));
                                fma2(h, F2(-1.f, -1.f), x).get(a, b);
                                lo[e] = cvt_bf16x2(a, b);
                            }
                            uint8_t* dst = ph + (j >> 3) * (kChunk * 16);
                            *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                            *reinterpret_cast<uint4*>(dst + L::kP) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        }
                    }
                if (masked && (kStream || wg == 0)) {
                    // Values of positions that some row does not see: behind the
                    // length they become zero (a weight of zero does not silence a
                    // NaN), between the rows' last positions non-finite ones do,
                    // and are added at the end to the rows that see them.
                    // (The slots' last V have been consumed: product_done.)
                    ok = ok && wait(&v_full[v0.at], v0.round, deadp);
                    if (kPieces == 2) ok = ok && wait(&v_full[v1.at], v1.round, deadp);
                    auto row = [&](int r) {
                        return vslots + (kPieces == 2 && r >= SPEC_PAGE ? v1.at : v0.at) * L::kPiece +
                               (kPieces == 2 ? r & (SPEC_PAGE - 1) : r) * 128;
                    };
                    if (kp >= w.len) {          // a thread's own row; lanes start at different banks
                        uint8_t* const z = row(key);
#pragma unroll
                        for (int hf = 0; hf < HD / 64; ++hf)
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                *reinterpret_cast<uint4*>(z + hf * kPieceRows * 128 + (((e + lane) & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    const int from = max(0, last0 + 1 - c * kChunk), to = min(kChunk, w.len - c * kChunk);
#pragma unroll 1
                    for (int t = from * (HD / 8) + key; t < to * (HD / 8); t += 128) {
                        const int e = t % (HD / 8);
                        uint4* const at = reinterpret_cast<uint4*>(row(t / (HD / 8)) + (e >> 3) * kPieceRows * 128 + ((e & 7) << 4));
                        uint4 x = *at;
                        uint32_t* y = &x.x;
                        bool hit = false;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if ((y[k] & 0x7F80u) == 0x7F80u) hit = true, y[k] &= 0xFFFF0000u;
                            if ((y[k] & 0x7F800000u) == 0x7F800000u) hit = true, y[k] &= 0xFFFFu;
                        }
                        if (hit) {
                            *at = x;
                            poison[par] = seg + 1;
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[kStream ? i & 1 : 0]);
            }
            // sums over the warp's keys, a span of rows at a time: lanes exchange halves
            // until lane r holds row r, then lanes of the same row are added
#pragma unroll
            for (int j = 0; j < NC; j += kSpan)
                if (j < rows) {
                    float x[kSpan];
#pragma unroll
                    for (int e = 0; e < kSpan; e += 2) l[(j + e) / 2].get(x[e], x[e + 1]);
#pragma unroll
                    for (int h = kSpan / 2; h >= 1; h >>= 1) {
                        const bool up = lane & h;
#pragma unroll
                        for (int e = 0; e < h; ++e) {
                            const float give = up ? x[e] : x[e + h], keep = up ? x[e + h] : x[e];
                            x[e] = keep + __shfl_xor_sync(0xffffffffu, give, h);
                        }
                    }
#pragma unroll
                    for (int h = kSpan; h < 32; h <<= 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], h);
                    if (lane < kSpan) xl[par][gi][qd][col0 + j + lane] = x[0];
                }
            __syncwarp();
            if (lane == 0) mbar_arrive(&l_full[par]);
        }
    } else {
        // ---------------- results: thread = head dimension ----------------
        if constexpr (L::kResultRegs < 128) regs_down<L::kResultRegs>();
        const int qd = warp & 3, d = qd * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(qd * 32) << 16);
        int i = 0;                              // the segment's first unit
#pragma unroll 1
        for (int seg = 0;; ++seg) {
            const Seg w = take(false);
            if (bar_any(kResultBar, 128, *deadp != 0) || w.units == 0) break;
            const int par = seg & 1, last0 = w.last0;
            const int ga = kStream ? i & 1 : 0; // the warpgroup of the first unit; the other has none in a segment of one
            const bool two = kStream && w.units > 1, whole = w.slot < 0;
            i += w.units;
            bool ok = wait(&l_full[par], (seg >> 1) & 1, deadp, plan::wait_rounds(w.units));
            if (d < w.R) {
                const int r = d;
                float ma = -nref[par][ga][r], la = xl[par][ga][0][r] + xl[par][ga][1][r] + xl[par][ga][2][r] + xl[par][ga][3][r];
                float fa = 1.f, fb = 0.f;
                if (two) {
                    const int gb = ga ^ (kGroups - 1);
                    const float mb = -nref[par][gb][r];
                    const float lb = xl[par][gb][0][r] + xl[par][gb][1][r] + xl[par][gb][2][r] + xl[par][gb][3][r];
                    const float m = fmaxf(ma, mb);
                    fa = ex2_approx(ma - m);
                    fb = ex2_approx(mb - m);
                    la = la * fa + lb * fb;
                    ma = m;
                }
                if (whole) {
                    const float inv = 1.f / la;
                    fa *= inv;
                    fb *= inv;
                } else {
                    p.part_ml[(size_t)w.slot * RP + r] = make_float2(ma, la);
                }
                weight[par][r] = {fa, fb};
            }
            named_bar_sync(kResultBar, 128);
            const bool bad = poison[par] == seg + 1;
            ok = ok && wait(&o_full[par], (seg >> 1) & 1, deadp);
            tc_fence_after();
            uint16_t* const out = p.out + (long long)w.row0 * p.out_stride + (long long)w.head * p.group * HD + d;
            float* const part = p.part_o + (size_t)(whole ? 0 : w.slot) * RP * HD + d;
            // rows whose O^T is in flight together (more would be more instructions than the cache likes)
            constexpr int kStep = kStack ? 8 : 16;
#pragma unroll 1
            for (int j0 = 0; j0 < w.R; j0 += kStep) {
                // the rows' O^T (both parts) of the first warpgroup, and of the other
                float o[kStep], x[kStep], y[kStep], z[kStep];
                const uint32_t at = lanes + 2 * RP + (kStream ? par * 2 + ga : par) * L::kO + j0;
                const uint32_t bt = lanes + 2 * RP + (par * 2 + (ga ^ 1)) * L::kO + j0;
                auto ld = [](uint32_t a, float* r) { if constexpr (kStep == 8) tmem_ld8_async(a, r); else tmem_ld16_async(a, r); };
                ld(at, o);
                if (kStack) ld(at + RP, x);
                if (two) {
                    ld(bt, y);
                    if (kStack) ld(bt + RP, z);
                }
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < kStep; ++e) {
                    const plan::Pair f = weight[par][j0 + e];
                    o[e] = (kStack ? o[e] + x[e] : o[e]) * f.x;
                    if (two) o[e] += (kStack ? y[e] + z[e] : y[e]) * f.y;
                }
                if (d < HD) {
                    if (bad)                    // of the positions that some row of the block sees and some does not
#pragma unroll 1
                        for (int t = max(last0 + 1, w.c0 * kChunk); t < min(last0 + tok[w.R - 1] + 1, (w.c0 + w.units) * kChunk); ++t) {
                            const int page = p.tables[(size_t)w.q * p.table_pages + t / SPEC_PAGE];
                            if (page < 0 || page >= p.num_pages) continue;
                            const float v = bf2f(p.vpool[(((size_t)page * p.hkv + w.head) * SPEC_PAGE + t % SPEC_PAGE) * HD + d]);
                            if (!isfinite(v))
#pragma unroll
                                for (int e = 0; e < kStep; ++e)
                                    if (t <= last0 + tok[j0 + e]) o[e] += v;
                        }
                    if (whole) {
                        if (last0 < 0) {        // rows without a position
#pragma unroll
                            for (int e = 0; e < kStep; ++e)
                                if (last0 + tok[j0 + e] < 0) o[e] = 0.f;
                        }
                        // (the offsets first: a guard around each load would wait for each)
#pragma unroll
                        for (int e0 = 0; e0 < kStep; e0 += 8) {
                            long long off[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) off[e] = col_off[j0 + e0 + e];
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (j0 + e0 + e < w.R) out[off[e]] = f2bf(o[e0 + e]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < kStep; ++e)
                            if (j0 + e < w.R) part[(j0 + e) * HD] = o[e];
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&o_empty[par]);
                mbar_arrive(&l_empty[par]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && dead && p.err) atomicCAS(p.err, 0, SPEC_PAGED_TIMEOUT);
    if (warp == kScoreWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kCols);
    }
}

// What the head layout has to satisfy; null when it does.
const char* head_error(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t max_new) {
    if (head_dim != 64 && head_dim != 128) return "spec_paged_attention: head_dim must be 64 or 128";
    if (n_kv_heads < 1 || n_kv_heads > 1024 || n_heads < n_kv_heads || n_heads % n_kv_heads)
        return "spec_paged_attention: n_heads must be a multiple of n_kv_heads, 1..1024";
    if (n_heads / n_kv_heads > 128) return "spec_paged_attention: at most 128 query heads per kv head";
    if (max_new < 1) return "spec_paged_attention: max_new must be at least 1";
    return nullptr;
}

// bf16 [d2][d1][d0] with strides s1, s2 (elements), read in boxes of [b2][b1][64], 128-byte swizzle.
bool encode(CUtensorMap* map, const void* p, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t s1, uint64_t s2, uint32_t b1,
            uint32_t b2) {
    const cuuint64_t dims[3] = {d0, d1, d2}, strides[2] = {s1 * 2, s2 * 2};
    const cuuint32_t box[3] = {64, b1, b2}, step[3] = {1, 1, 1};
    return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, step,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD, int RP>
cudaError_t run(PagedParams& p, int ctas, cudaStream_t s) {
    const void* fn = (const void*)paged_attn_kernel<HD, RP>;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Plan<HD, RP>::kBytes);
    if (e != cudaSuccess) return e;
    void* args[] = {&p};
    if ((e = launch(fn, dim3((unsigned)ctas), kThreads, Plan<HD, RP>::kBytes, s, args)) != cudaSuccess || p.whole) return e;
    int rp = RP;
    void* jargs[] = {static_cast<PagedCommon*>(&p), &rp};
    return launch((const void*)paged_join_kernel<HD>, dim3((unsigned)ctas, 2 * (RP <= 16 ? 1 : RP / 16)), 32 * kJoinWarps, 0, s, jargs);
}

}  // namespace
}  // namespace sv

extern "C" {

using namespace sv;

spec_status spec_paged_attention_workspace(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t max_new,
                                           int32_t table_pages, size_t* out_bytes) {
    if (!out_bytes) return bad("spec_paged_attention_workspace: null pointer");
    if (const char* e = head_error(n_heads, n_kv_heads, head_dim, max_new)) return bad(e);
    if (table_pages < 1 || table_pages > SPEC_MAX_TABLE) return bad("spec_paged_attention: table_pages must be in 1..1048576");
    if (split::whole_pairs(table_pages)) {
        *out_bytes = 0;
        return SPEC_OK;
    }
    const int sms = current_sms();
    if (!sms) {
        set_last_error("spec_paged_attention_workspace: no current CUDA device");
        return SPEC_ERR_CUDA;
    }
    *out_bytes = Work(sms, split::tile_rows(n_heads / n_kv_heads, max_new), head_dim).bytes;
    return SPEC_OK;
}

spec_status spec_paged_attention(const void* d_q, int64_t q_stride, const int32_t* d_row_start, const int32_t* d_len,
                                 const int32_t* d_tables, int32_t table_pages, int32_t nseq, int32_t rows,
                                 int32_t max_new, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, float scale,
                                 const void* d_kpool, const void* d_vpool, int32_t num_pages, void* d_out,
                                 int64_t out_stride, int32_t* d_error_opt, void* d_work, size_t work_bytes,
                                 void* cuda_stream) {
    if (const char* e = head_error(n_heads, n_kv_heads, head_dim, max_new)) return bad(e);
    if (nseq < 0 || nseq > SPEC_MAX_SEQS) return bad("spec_paged_attention: nseq must be in 0..1024");
    if (rows < 0) return bad("spec_paged_attention: negative rows");
    if (table_pages < 1 || table_pages > SPEC_MAX_TABLE) return bad("spec_paged_attention: table_pages must be in 1..1048576");
    if (num_pages < 1 || num_pages > SPEC_MAX_PAGES) return bad("spec_paged_attention: num_pages must be in 1..33554431");
    if ((int64_t)num_pages * n_kv_heads > 0x7fffffff) return bad("spec_paged_attention: num_pages * n_kv_heads must fit int32");
    if (!(scale > 0.f) || !isfinite(scale)) return bad("spec_paged_attention: scale must be positive and finite");
    const int64_t row = (int64_t)n_heads * head_dim;
    if (q_stride < row || out_stride < row || (q_stride & 7) || (out_stride & 7) || q_stride >= (1ll << 38) ||
        out_stride >= (1ll << 38))
        return bad("spec_paged_attention: row strides must be multiples of 8, at least n_heads * head_dim and below 2^38");
    if (nseq == 0 || rows == 0) return SPEC_OK;
    const bool whole = split::whole_pairs(table_pages);
    if (!d_q || !d_row_start || !d_len || !d_tables || !d_kpool || !d_vpool || !d_out || (!whole && !d_work))
        return bad("spec_paged_attention: null pointer");
    if (misaligned(d_q, 16) || misaligned(d_out, 16) || misaligned(d_kpool, 16) || misaligned(d_vpool, 16))
        return bad("spec_paged_attention: queries, output and pools must be 16-byte aligned");
    if (misaligned(d_row_start, 4) || misaligned(d_len, 4) || misaligned(d_tables, 4) || misaligned(d_error_opt, 4))
        return bad("spec_paged_attention: an int32 pointer is not 4-byte aligned");
    if (misaligned(d_work, 256)) return bad("spec_paged_attention: d_work is not 256-byte aligned");
    const int group = n_heads / n_kv_heads, rp = split::tile_rows(group, max_new), tokens = rp / group;
    // every unit has to fit int32, whatever the lengths on the device
    const int64_t pairs = ((int64_t)nseq + rows / tokens) * n_kv_heads;
    if (pairs > 0x7fffffffll / ((table_pages + 1) / 2))
        return bad("spec_paged_attention: too much work for one call ((nseq + rows / tile) * n_kv_heads * table_pages / 2)");
    if (!whole && work_bytes < Work(1, rp, head_dim).bytes) return bad("spec_paged_attention: work_bytes is less than these heads need");
    const int sms = current_sms();
    if (!sms) {
        set_last_error("spec_paged_attention: no current CUDA device");
        return SPEC_ERR_CUDA;
    }
    const Work work(sms, rp, head_dim);
    if (!whole && work_bytes < work.bytes) return bad("spec_paged_attention: work_bytes is less than these heads need");
    if (!encode_fn()) {
        set_last_error("spec_paged_attention: the driver has no cuTensorMapEncodeTiled");
        return SPEC_ERR_CUDA;
    }
    PagedParams p;
    const uint64_t page = (uint64_t)SPEC_PAGE * head_dim;
    if (!encode(&p.mq, d_q, head_dim, n_heads, rows, head_dim, q_stride, group, tokens) ||
        !encode(&p.mk, d_kpool, head_dim, SPEC_PAGE, (uint64_t)num_pages * n_kv_heads, head_dim, page, SPEC_PAGE, 1) ||
        !encode(&p.mv, d_vpool, head_dim, SPEC_PAGE, (uint64_t)num_pages * n_kv_heads, head_dim, page, SPEC_PAGE, 1)) {
        set_last_error("spec_paged_attention: a tensor map could not be made");
        return SPEC_ERR_CUDA;
    }
    p.row_start = d_row_start;
    p.len = d_len;
    p.tables = d_tables;
    p.table_pages = table_pages;
    p.nseq = nseq;
    p.rows = rows;
    p.hkv = n_kv_heads;
    p.group = group;
    p.tokens = tokens;
    p.whole = whole;
    p.scale_log2 = scale * 1.44269504088896340736f;
    p.vpool = static_cast<const uint16_t*>(d_vpool);
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
        e = rp == 16 ? run<128, 16>(p, sms, s) : rp == 32 ? run<128, 32>(p, sms, s) : rp == 64 ? run<128, 64>(p, sms, s)
                                                                                         : run<128, 128>(p, sms, s);
    else
        e = rp == 16 ? run<64, 16>(p, sms, s) : rp == 32 ? run<64, 32>(p, sms, s) : rp == 64 ? run<64, 64>(p, sms, s)
                                                                                       : run<64, 128>(p, sms, s);
    return e == cudaSuccess ? SPEC_OK : failed(e);
}

}  // extern "C"
