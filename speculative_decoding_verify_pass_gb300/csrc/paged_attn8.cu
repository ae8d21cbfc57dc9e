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
//                       parts lie one behind the other along the product's k.
//     P^T = exp2(2^(a + ek) scale log2e S^T - m)    ek: the key's scale
//     O^T += V8^T P'^T  P' = 2^(ev - r + 8) P, three e5m2 parts      ev: the value's scale
// A value's scale goes into its weight, relative to r, the largest scale seen, so
// that the codes enter the product as they are.  Weights need more range than bits
// (a key far down still counts when there are 100000 like it), so their parts are
// e5m2: 3 significant bits each, 9 together, and 2^-17 to 57344 where e4m3 ends at
// 2^-10 and 448.  Relative to the reference's weight, what is lost lies below 2^-25.
//
// That range is what decides the softmax's references: a weight may exceed its row's
// reference by 2^7.75 only (fp32 and bf16 bear 2^40).  So a row takes the maximum of
// its segment's first chunk (redux over each warp's 32 keys), and r that chunk's
// largest scale; when a later score or scale exceeds them, row references, sums and O^T
// move to the chunk's.
//
// Roles, by warpgroup: 0 and 1 softmax (thread = key); 2 one warp each for the MMAs of
// S^T, those of O^T, the copies of V, and the list of segments with the copies of K
// and the scales; 3 splits the next segment's queries into their parts, then writes
// this segment's results (thread = head dimension).
#include <stdio.h>

#include "paged_core.cuh"
#include "paged_plan8.h"

namespace sv {
namespace {

using plan8::kParts;
using plan8::kScaleSlots;
using plan8::Plan;

constexpr float kLimit8 = 7.75f;        // log2 by which a weight, its value's scale included, may exceed the references
constexpr int kShift8 = 8;              // weights are kept times 2^8: 2^(8 + 7.75) is below e5m2's 57344
constexpr int kFarScale = 60;           // a scale this far above the reference moves it: 2^60 times a small weight still is one

struct Paged8Params : PagedCommon {
    CUtensorMap mk, mv;
    const uint16_t* q;
    long long q_stride;
    const uint8_t *vpool, *scales;
};

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
// The next e5m2 part of two halves (an e5m2 code is a half's upper byte), and what it leaves.
__device__ __forceinline__ uint32_t part_e5m2(uint32_t& h) {
    uint16_t c;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(c) : "r"(h));
    uint32_t t;
    asm("prmt.b32 %0, %1, 0, 0x1404;" : "=r"(t) : "r"((uint32_t)c));
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(h) : "r"(t));
    return c;
}
__device__ __forceinline__ uint32_t last_e5m2(uint32_t h) {
    uint16_t c;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(c) : "r"(h));
    return c;
}
__device__ __forceinline__ uint32_t cvt_f16x2(F2 x) {
    float a, b;
    x.get(a, b);
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

template <int HD, int RP>
__global__ void __block_size__((kThreads, 1, 1)) __maxnreg__(128) paged_attn8_kernel(const __grid_constant__ Paged8Params p) {
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
    extern __shared__ uint8_t smem_raw[];
    __shared__ plan8::Fixed<RP> sh;

    uint8_t* base = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* kslots = base;
    uint8_t* vslots = kslots + NK * L::kSlot;
    uint8_t* qs = vslots + NV * L::kSlot + L::kPad;
    uint8_t* ps = qs + NQ * L::kQ;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < NK; ++i) {
            mbar_init(&sh.k_full[i], 1);
            mbar_init(&sh.k_empty[i], 1);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(&sh.v_full[i], 1);
            mbar_init(&sh.v_empty[i], 1);
        }
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(&sh.c_full[i], 1);
            mbar_init(&sh.c_empty[i], kArrive);
        }
        for (int i = 0; i < NQ; ++i) {
            mbar_init(&sh.q_full[i], 4);
            mbar_init(&sh.q_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.r_full[i], 4);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_empty[i], kArrive);
            mbar_init(&sh.o_full[i], 1);
            mbar_init(&sh.o_empty[i], 4);
            mbar_init(&sh.l_full[i], kSoftWarps);
            mbar_init(&sh.l_empty[i], 4);
            mbar_init(&sh.fin[i], 1);
            sh.poison[i] = 0;
        }
        for (int i = 0; i < NP; ++i) {
            mbar_init(&sh.p_full[i], kArrive);
            mbar_init(&sh.p_empty[i], 1);
        }
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(&sh.seg_full[i], 1);
            mbar_init(&sh.seg_empty[i], kReaders);
        }
        fence_barrier_init();
        sh.dead = 0;
        sh.first[0] = 0;
    }
#pragma unroll 1
    for (int i = tid; i < RP; i += kThreads) {
        const int t = i / p.group;
        sh.tok[i] = t;
        sh.col_off[i] = t * p.out_stride + (long long)(i - t * p.group) * HD;
    }
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
    volatile int* deadp = &sh.dead;
    Ring<kSegs> sr;                             // every role's place in the list of segments
    auto take = [&](bool one) {                 // the next segment; `one`: this thread alone stands for its warp
        wait(&sh.seg_full[sr.at], sr.round, deadp);
        const Seg s = sh.segs[sr.at];
        if (!one) __syncwarp();
        if (one || lane == 0) mbar_arrive(&sh.seg_empty[sr.at]);
        sr.step();
        return s;
    };

    if (warp >= kScoreWarp && warp < kResultWarp) {
        regs_down<L::kIssueRegs>();
        if (warp == kLoadKWarp) {
            // ---------------- the list of segments, K and scale copies, and what the join kernel has to do here ----------------
            const bool few = p.nseq <= kFewSeqs;
            Walk w(p, sh.first, few ? sh.few_start : p.row_start, few ? sh.few_len : p.len, begin, end);
            Meta into = {}, from = {};
            Ring<NK> kr;
            Ring<kScaleSlots> cr;
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
                ok = __all_sync(0xffffffffu, wait(&sh.seg_empty[sr.at], sr.round ^ 1, deadp));
                if (!ok) break;
                if (lane == 0) {
                    sh.segs[sr.at] = s;
                    mbar_arrive(&sh.seg_full[sr.at]);
                }
                sr.step();
                if (!more) break;
                PageWalk pages;
#pragma unroll 1
                for (int k = 0; k < s.units; ++k) {
                    pages.at(p, s, k, lane);
                    ok = __all_sync(0xffffffffu, wait(&sh.c_empty[cr.at], cr.round ^ 1, deadp) && wait(&sh.k_empty[kr.at], kr.round ^ 1, deadp));
                    if (!ok) break;
                    if (elect_one()) {
                        uint64_t* cf = &sh.c_full[cr.at];
                        // a bad page (it reads as zeros) has no scales: ones
                        const bool c0 = pages.count > 0 && pages.z0 >= 0, c1 = pages.count > 1 && pages.z1 >= 0;
                        if (pages.count > 0 && !c0)
                            for (int i = 0; i < 8; ++i) reinterpret_cast<uint4*>(sh.scale[cr.at][0])[i] = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                        if (pages.count > 1 && !c1)
                            for (int i = 0; i < 8; ++i) reinterpret_cast<uint4*>(sh.scale[cr.at][1])[i] = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                        fence_proxy_async_smem();
                        mbar_arrive_expect_tx(cf, (c0 ? 2 * SPEC_PAGE : 0) + (c1 ? 2 * SPEC_PAGE : 0));
                        if (c0) bulk_g2s(sh.scale[cr.at][0], p.scales + (size_t)pages.z0 * 2 * SPEC_PAGE, 2 * SPEC_PAGE, cf);
                        if (c1) bulk_g2s(sh.scale[cr.at][1], p.scales + (size_t)pages.z1 * 2 * SPEC_PAGE, 2 * SPEC_PAGE, cf);
                        uint64_t* full = &sh.k_full[kr.at];
                        uint8_t* dst = kslots + kr.at * L::kSlot;
                        mbar_arrive_expect_tx(full, (uint32_t)(pages.count * SPEC_PAGE * HD));
                        if (pages.count > 0) tma3(dst, &p.mk, 0, 0, pages.z0, full);
                        if (pages.count > 1) tma3(dst + SPEC_PAGE * HD, &p.mk, 0, 0, pages.z1, full);
                    }
                    __syncwarp();
                    kr.step();
                    cr.step();
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
                for (int i = 0; i < NK; ++i) drain(&sh.k_full[i], i < kr.at ? kr.round : kr.round ^ 1);
#pragma unroll 1
                for (int i = 0; i < kScaleSlots; ++i) drain(&sh.c_full[i], i < cr.at ? cr.round : cr.round ^ 1);
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
                for (int k = 0; k < s.units; ++k) {
                    pages.at(p, s, k, lane);
                    ok = __all_sync(0xffffffffu, wait(&sh.v_empty[vr.at], vr.round ^ 1, deadp));
                    if (!ok) break;
                    if (elect_one()) {
                        uint64_t* full = &sh.v_full[vr.at];
                        uint8_t* dst = vslots + vr.at * L::kSlot;
                        mbar_arrive_expect_tx(full, (uint32_t)(pages.count * SPEC_PAGE * HD));
                        if (pages.count > 0) tma3(dst, &p.mv, 0, 0, pages.z0, full);
                        if (pages.count > 1) tma3(dst + SPEC_PAGE * HD, &p.mv, 0, 0, pages.z1, full);
                    }
                    __syncwarp();
                    vr.step();
                }
                if (!ok) break;
            }
            if (lane == 0 && *deadp) {
#pragma unroll 1
                for (int i = 0; i < NV; ++i) drain(&sh.v_full[i], i < vr.at ? vr.round : vr.round ^ 1);
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
                    ok = wait(&sh.q_full[qr.at], qr.round, deadp);
                    const uint32_t id = idesc8(128, (s.R + 15) & ~15, 0, 0);
                    const uint32_t dq = lo_desc(qa + qr.at * L::kQ, 16);
                    constexpr uint32_t kHi = hi_swizzled<HD>(8 * HD);
#pragma unroll 1
                    for (int k = 0; k < s.units && ok; ++k) {
                        ok = wait(&sh.k_full[ks.at], ks.round, deadp) && wait(&sh.s_empty[sb.at], sb.round ^ 1, deadp);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t dk = lo_desc(sa + ks.at * L::kSlot, 16);
#pragma unroll
                        for (int part = 0; part < 2; ++part)
#pragma unroll
                            for (int e = 0; e < HD / 32; ++e)
                                umma8_lo(tmem + sb.at * RP, dk + e * 2, kHi, dq + part * (L::kQPart >> 4) + e * 2, kHi, id, (part | e) != 0);
                        umma_commit(&sh.s_full[sb.at]);
                        umma_commit(&sh.k_empty[ks.at]);
                        ks.step();
                        sb.step();
                    }
                    if (ok) umma_commit(&sh.q_empty[qr.at]);
                    qr.step();
                }
                if (!ok || *deadp) {
                    umma_commit(&sh.fin[0]);
                    drain(&sh.fin[0], 0);
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
                    ok = wait(&sh.o_empty[seg & 1], ((seg >> 1) & 1) ^ 1, deadp);
                    // A = V^T and B = P^T, both MN-major
                    const uint32_t id = idesc8(128, kStack ? kParts * RP : (s.R + 15) & ~15, 0, 1) | (1u << 15) | (1u << 16);
#pragma unroll 1
                    for (int k = 0; k < s.units && ok; ++k, ++j) {
                        ok = wait(&sh.p_full[pr.at], pr.round, deadp) && wait(&sh.v_full[vs.at], vs.round, deadp);
                        if (!ok) break;
                        tc_fence_after();
                        // P^T: core matrices of 16 rows (of the product's N) x 8 keys, 128 bytes apart along the keys
                        const uint32_t dp = lo_desc(pa + pr.at * kParts * L::kP, 128);
                        const uint32_t dv = lo_desc(sa + vs.at * L::kSlot, 1024);
                        constexpr uint32_t kHiV = hi_swizzled<HD>(8 * HD), kHiP = (kChunk * 16 >> 4) | (1u << 14);
                        const int og = kStream ? (seg & 1) * 2 + (j & 1) : seg & 1;
                        const uint32_t o = tmem + 2 * RP + og * L::kO;
                        const bool more = k >= kGroups;     // this O^T holds earlier chunks
#pragma unroll
                        for (int part = 0; part < (kStack ? 1 : kParts); ++part)
#pragma unroll
                            for (int e = 0; e < kChunk / 32; ++e)
                                umma8_lo(o, dv + e * (32 * HD >> 4), kHiV, dp + part * (L::kP >> 4) + e * (32 * 16 >> 4), kHiP, id,
                                         more || (part | e) != 0);
                        umma_commit(&sh.v_empty[vs.at]);
                        umma_commit(&sh.p_empty[pr.at]);
                        vs.step();
                        pr.step();
                    }
                    if (ok) umma_commit(&sh.o_full[seg & 1]);
                }
                if (!ok || *deadp) {
                    umma_commit(&sh.fin[1]);
                    drain(&sh.fin[1], 0);
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
        Ring<kScaleSlots> cs;                   // and of its scales
        bool ok = true;
#pragma unroll 1
        for (int seg = 0;; ++seg) {
            const Seg w = take(false);
            if (bar_any(bar, 128, *deadp != 0) || w.units == 0) break;   // after a wait that gave up, all of the warpgroup leaves
            const int par = seg & 1, last0 = w.last0, rows = w.R - col0;   // live rows of this thread
            float* const mine = sh.nref[par][gi];
            const float* const qmul = sh.qmul[par];
            ok = ok && wait(&sh.l_empty[par], ((seg >> 1) & 1) ^ 1, deadp);   // the results of two segments ago have been read
            ok = ok && wait(&sh.r_full[par], (seg >> 1) & 1, deadp);          // the query rows' powers of two are there
            F2 l[NC / 2];
#pragma unroll
            for (int j = 0; j < NC / 2; ++j) l[j] = F2(0.f, 0.f);
            bool fresh = true, wide = false;    // wide: a reference past 2^24, every chunk takes rounded products
            int vref = 0;                       // scale byte that O^T is relative to
#pragma unroll 1
            for (int c = w.c0; c < w.c0 + w.units; ++c, ++i) {
                const Ring<NV> v0 = vs;         // the chunk's V
                vs.step();
                const Ring<kScaleSlots> c0 = cs;
                cs.step();
                if (kStream && (i & 1) != wg) continue;
                const uint32_t st = lanes + (i & 1) * RP + col0;
                const int kp = c * kChunk + key;
                const bool masked = (c + 1) * kChunk - 1 > last0;   // some row does not see all of the chunk
                ok = ok && wait(&sh.c_full[c0.at], c0.round, deadp);
                int kb = sh.scale[c0.at][key >> 6][0][key & 63], vb = sh.scale[c0.at][key >> 6][1][key & 63];
                if (kp >= w.len) kb = 127, vb = 0;      // no position: whatever stands there
                const bool nan = kb == 255 || vb == 255;
                if (nan) kb = 127, vb = 0;
                const float km = scale_of(kb);
                const F2 km2(km, km);
                ok = ok && wait(&sh.s_full[i & 1], (i >> 1) & 1, deadp);
                tc_fence_after();
                float s[NC];
                // this thread's P^T buffer is free (and its rows' O^T complete) once their last product is
                auto product_done = [&]() {
                    ok = ok && wait(&sh.p_empty[kStream ? i & 1 : 0], ((kStream ? i >> 1 : i) & 1) ^ 1, deadp);
                };
                // the chunk's products, NaN under a scale that is none, -inf where a row does not see the key
                auto load = [&]() {
#pragma unroll
                    for (int j = 0; j < NC; j += kSpan)
                        if (j < rows) {
                            if constexpr (kSpan == 8) tmem_ld8_async(st + j, s + j);
                            else if constexpr (kSpan == 16) tmem_ld16_async(st + j, s + j);
                            else tmem_ld32_async(st + j, s + j);
                        }
                    tmem_wait_ld();
                    if (nan) {
#pragma unroll
                        for (int j = 0; j < NC; ++j) s[j] = __uint_as_float(0x7FC00000u);
                    }
                    if (masked) {
                        // rows are in token order: the key is hidden from the tokens before it
                        const int hidden = min(max(kp - last0, 0), RP) * p.group - col0;
#pragma unroll
                        for (int j = 0; j < NC; ++j)
                            if (j < hidden) s[j] = -INFINITY;
                    }
                };
                load();
                if (rows > 0) {
                    bool move = fresh || wide;
                    if (!move) {
                        float top[2] = {kNone, kNone};
#pragma unroll
                        for (int j0 = 0; j0 < NC; j0 += kSpan)
                            if (j0 < rows) {
#pragma unroll
                                for (int j = j0; j < j0 + kSpan; j += 4) {
                                    const float4 m = *reinterpret_cast<const float4*>(&mine[col0 + j]);
                                    const float4 f = *reinterpret_cast<const float4*>(&qmul[col0 + j]);
                                    fma2(mul2(F2(s[j], s[j + 1]), km2), F2(f.x, f.y), F2(m.x, m.y)).get(s[j], s[j + 1]);
                                    fma2(mul2(F2(s[j + 2], s[j + 3]), km2), F2(f.z, f.w), F2(m.z, m.w)).get(s[j + 2], s[j + 3]);
                                    top[j / 4 & 1] = fmaxf(top[j / 4 & 1], fmaxf(fmaxf(s[j], s[j + 1]), fmaxf(s[j + 2], s[j + 3])));
                                }
                            }
                        const float above = fmaxf(top[0], top[1]);
                        move = bar_any(bar, 128, above + (float)max(vb - vref, 0) > kLimit8 && above > -1e30f || vb - vref > kFarScale);
                        if (move) load();
                    }
                    if (move) {
                        // The references move up to the chunk's maxima (a first chunk's become
                        // them), the sums and O^T with them.  So that a reference and the score
                        // that it comes from cancel whatever their size, the scores are here
                        // rounded products, as it is: the fused product of a score past 2^24
                        // differs from it by powers of two, past 2^31 by more than a weight can hold.
                        float (*const mx)[RP] = sh.xl[par][gi];
#pragma unroll
                        for (int j0 = 0; j0 < NC; j0 += kSpan)
                            if (j0 < rows) {
                                float keep = 0.f;
#pragma unroll
                                for (int j = j0; j < j0 + kSpan; j += 4) {
                                    const float4 f = *reinterpret_cast<const float4*>(&qmul[col0 + j]);
                                    mul2(mul2(F2(s[j], s[j + 1]), km2), F2(f.x, f.y)).get(s[j], s[j + 1]);
                                    mul2(mul2(F2(s[j + 2], s[j + 3]), km2), F2(f.z, f.w)).get(s[j + 2], s[j + 3]);
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        const float m = warp_max(s[j + e]);
                                        if (lane == ((j + e) & (kSpan - 1))) keep = m;
                                    }
                                }
                                if (lane < kSpan) mx[qd][col0 + j0 + lane] = keep;
                            }
                        const int vt = __reduce_max_sync(0xffffffffu, vb);
                        if (lane == 0) sh.vtop[wg][qd] = vt;
                        if (!fresh) {
                            product_done();
                            tc_fence_after();
                        }
                        named_bar_sync(bar, 128);
                        const int vnow = max(max(max(sh.vtop[wg][0], sh.vtop[wg][1]), max(sh.vtop[wg][2], sh.vtop[wg][3])), fresh ? 0 : vref);
                        float now = 0.f;
                        if (key < NC) {         // one thread per row: the new reference, and what the old weights shrink by
                            const int r = col0 + key;
                            const float m = fmaxf(fmaxf(mx[0][r], mx[1][r]), fmaxf(mx[2][r], mx[3][r]));
                            const float old = fresh ? kNone : -mine[r];
                            now = key < rows ? fmaxf(old, m) : INFINITY;      // rows past R weigh nothing
                            mine[r] = -now;
                            mx[0][r] = key < rows ? ex2_approx(old - now) : 0.f;
                        }
                        if (key == 0) sh.vref[par][wg] = vnow;
                        wide = bar_any(bar, 128, key < rows && fabsf(now) > kWide && now > kNone);
                        if (!fresh) {
                            const float vshrink = scale_of(max(vref - vnow + 127, 0));      // 1 or less
#pragma unroll
                            for (int j = 0; j < NC; j += 2) {
                                float x, y;
                                l[j / 2].get(x, y);
                                l[j / 2] = F2(x * mx[0][col0 + j], y * mx[0][col0 + j + 1]);
                            }
                            const uint32_t ot = lanes + 2 * RP + (kStream ? par * 2 + wg : par) * L::kO + col0;
#pragma unroll 1
                            for (int j = 0; j < (kStack ? kParts * NC : NC); j += 8)   // stacked: the other parts' columns follow
                                if ((kStack ? j & (NC - 1) : j) < rows) {
                                    float o[8];
                                    tmem_ld8_async(ot + j, o);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int e = 0; e < 8; ++e) o[e] *= mx[0][col0 + (j & (NC - 1)) + e] * vshrink;
                                    tmem_st8(ot + j, o);
                                }
                            tmem_wait_st();
                        }
                        vref = vnow;
#pragma unroll
                        for (int j0 = 0; j0 < NC; j0 += kSpan)
                            if (j0 < rows) {
#pragma unroll
                                for (int j = j0; j < j0 + kSpan; j += 4) {
                                    const float4 m = *reinterpret_cast<const float4*>(&mine[col0 + j]);
                                    add2(F2(s[j], s[j + 1]), F2(m.x, m.y)).get(s[j], s[j + 1]);
                                    add2(F2(s[j + 2], s[j + 3]), F2(m.z, m.w)).get(s[j + 2], s[j + 3]);
                                }
                            }
                        if (!fresh) named_bar_sync(bar, 128);   // everyone has read mx
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sh.s_empty[i & 1]);
                    mbar_arrive(&sh.c_empty[c0.at]);
                }
                fresh = false;
                const int ve = vb - vref + kShift8 + 127;
                const float vm = __uint_as_float((uint32_t)min(max(ve, 0), 254) << 23);
                const F2 vm2(vm, vm);
                product_done();
                uint8_t* ph = ps + (kStream ? i & 1 : 0) * kParts * L::kP + (col0 >> 4) * (kChunk * 16) + key * 16;
#pragma unroll
                for (int j0 = 0; j0 < NC; j0 += kSpan)
                    if (j0 < rows) {
#pragma unroll
                        for (int j = j0; j < j0 + kSpan; j += 8) {
                            uint32_t c1[4], c2[4], c3[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const F2 x(ex2_approx(s[j + 2 * e]), ex2_approx(s[j + 2 * e + 1]));
                                l[j / 2 + e] = add2(l[j / 2 + e], x);
                                uint32_t h = cvt_f16x2(mul2(x, vm2));
                                c1[e] = part_e5m2(h);
                                c2[e] = part_e5m2(h);
                                c3[e] = last_e5m2(h);
                            }
                            uint8_t* dst = ph + (j >> 4) * (kChunk * 16) + (j & 8);
                            *reinterpret_cast<uint2*>(dst) = make_uint2(c1[0] | c1[1] << 16, c1[2] | c1[3] << 16);
                            *reinterpret_cast<uint2*>(dst + L::kP) = make_uint2(c2[0] | c2[1] << 16, c2[2] | c2[3] << 16);
                            *reinterpret_cast<uint2*>(dst + 2 * L::kP) = make_uint2(c3[0] | c3[1] << 16, c3[2] | c3[3] << 16);
                        }
                    }
                if (masked && (kStream || wg == 0)) {
                    // Values of positions that some row does not see: behind the
                    // length they become zero (a weight of zero does not silence a
                    // NaN), between the rows' last positions NaN do, and are added at
                    // the end to the rows that see them.
                    // (The slot's last V has been consumed: product_done.)
                    ok = ok && wait(&sh.v_full[v0.at], v0.round, deadp);
                    uint8_t* const tile = vslots + v0.at * L::kSlot;
                    if (kp >= w.len) {          // a thread's own row; lanes start at different banks
#pragma unroll
                        for (int e = 0; e < HD / 16; ++e)
                            *reinterpret_cast<uint4*>(tile + key * HD + (((e + lane) & (HD / 16 - 1)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    const int from = max(0, last0 + 1 - c * kChunk), to = min(kChunk, w.len - c * kChunk);
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
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_full[kStream ? i & 1 : 0]);
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
                    if (lane < kSpan) sh.xl[par][gi][qd][col0 + j + lane] = x[0];
                }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.l_full[par]);
        }
    } else {
        // ---------------- the next segment's queries, and results: thread = head dimension ----------------
        if constexpr (L::kResultRegs < 128) regs_down<L::kResultRegs>();
        const int qd = warp & 3, d = qd * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(qd * 32) << 16);
        Ring<NQ> qr;
        // Queries in two e4m3 parts with a power of two for each row, 8 elements a thread.
        auto split_queries = [&](const Seg& s, int par) {
            constexpr int kRowThreads = HD / 8, kPass = 128 / kRowThreads;
            bool ok = wait(&sh.q_empty[qr.at], qr.round ^ 1, deadp);
            uint8_t* const tile = qs + qr.at * L::kQ;
            const int b = d & (kRowThreads - 1);
#pragma unroll 1
            for (int r0 = 0; r0 < s.R; r0 += kPass) {
                const int r = r0 + d / kRowThreads, t = sh.tok[min(r, s.R - 1)];
                uint4 x = {};
                if (r < s.R)
                    x = *reinterpret_cast<const uint4*>(p.q + (long long)(s.row0 + t) * p.q_stride +
                                                        (long long)(s.head * p.group + r - t * p.group) * HD + b * 8);
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
            if (lane == 0) {
                mbar_arrive(&sh.q_full[qr.at]);
                mbar_arrive(&sh.r_full[par]);
            }
            qr.step();
            return ok;
        };
        int i = 0;                              // the segment's first unit
        Seg next = take(false);
        bool gone = bar_any(kResultBar, 128, *deadp != 0);
        if (!gone && next.units) split_queries(next, 0);
#pragma unroll 1
        for (int seg = 0; !gone && next.units; ++seg) {
            const Seg w = next;
            next = take(false);
            gone = bar_any(kResultBar, 128, *deadp != 0);
            if (gone) break;
            if (next.units) split_queries(next, (seg + 1) & 1);
            const int par = seg & 1, last0 = w.last0;
            const int ga = kStream ? i & 1 : 0; // the warpgroup of the first unit; the other has none in a segment of one
            const bool two = kStream && w.units > 1, whole = w.slot < 0;
            i += w.units;
            bool ok = wait(&sh.l_full[par], (seg >> 1) & 1, deadp, plan::wait_rounds(w.units));
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
                if (whole) {
                    const float inv = 1.f / la;
                    fa *= inv;
                    fb *= inv;
                } else {
                    p.part_ml[(size_t)w.slot * RP + r] = make_float2(ma, la);
                }
                // O^T is in units of 2^(r - 8), r the warpgroup's that formed the row's weights
                fa = fa * (1.f / (1 << kShift8)) * scale_of(sh.vref[par][kStream ? ga : r / NC]);
                if (two) fb = fb * (1.f / (1 << kShift8)) * scale_of(sh.vref[par][ga ^ 1]);
                sh.weight[par][r] = {fa, fb};
            }
            named_bar_sync(kResultBar, 128);
            const bool bad = sh.poison[par] == seg + 1;
            ok = ok && wait(&sh.o_full[par], (seg >> 1) & 1, deadp);
            tc_fence_after();
            uint16_t* const out = p.out + (long long)w.row0 * p.out_stride + (long long)w.head * p.group * HD + d;
            float* const part = p.part_o + (size_t)(whole ? 0 : w.slot) * RP * HD + d;
            // rows whose O^T is in flight together (more would be more instructions than the cache likes)
            constexpr int kStep = kStack ? 8 : 16;
#pragma unroll 1
            for (int j0 = 0; j0 < w.R; j0 += kStep) {
                // the rows' O^T of the first warpgroup, and of the other
                float o[kStep], y[kStep];
                const uint32_t at = lanes + 2 * RP + (kStream ? par * 2 + ga : par) * L::kO + j0;
                const uint32_t bt = lanes + 2 * RP + (par * 2 + (ga ^ 1)) * L::kO + j0;
                auto ld = [](uint32_t a, float* r) {
                    if constexpr (kStack) {     // its three parts
                        float u[kStep], v[kStep];
                        tmem_ld8_async(a, r);
                        tmem_ld8_async(a + RP, u);
                        tmem_ld8_async(a + 2 * RP, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < kStep; ++e) r[e] += u[e] + v[e];
                    } else {
                        tmem_ld16_async(a, r);
                        tmem_wait_ld();
                    }
                };
                ld(at, o);
                if (two) ld(bt, y);
#pragma unroll
                for (int e = 0; e < kStep; ++e) {
                    const plan::Pair f = sh.weight[par][j0 + e];
                    o[e] *= f.x;
                    if (two) o[e] += y[e] * f.y;
                }
                if (d < HD) {
                    if (bad)                    // of the positions that some row of the block sees and some does not
#pragma unroll 1
                        for (int t = max(last0 + 1, w.c0 * kChunk); t < min(last0 + sh.tok[w.R - 1] + 1, (w.c0 + w.units) * kChunk); ++t) {
                            const int page = p.tables[(size_t)w.q * p.table_pages + t / SPEC_PAGE];
                            if (page < 0 || page >= p.num_pages) continue;
                            const int code = p.vpool[(((size_t)page * p.hkv + w.head) * SPEC_PAGE + t % SPEC_PAGE) * HD + d];
                            if ((code & 0x7F) == 0x7F)
#pragma unroll
                                for (int e = 0; e < kStep; ++e)
                                    if (t <= last0 + sh.tok[j0 + e]) o[e] = __uint_as_float(0x7FC00000u);
                        }
                    if (whole) {
                        if (last0 < 0) {        // rows without a position
#pragma unroll
                            for (int e = 0; e < kStep; ++e)
                                if (last0 + sh.tok[j0 + e] < 0) o[e] = 0.f;
                        }
                        // (the offsets first: a guard around each load would wait for each)
#pragma unroll
                        for (int e0 = 0; e0 < kStep; e0 += 8) {
                            long long off[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) off[e] = sh.col_off[j0 + e0 + e];
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
                mbar_arrive(&sh.o_empty[par]);
                mbar_arrive(&sh.l_empty[par]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && sh.dead && p.err) atomicCAS(p.err, 0, SPEC_PAGED_TIMEOUT);
    if (warp == kScoreWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kCols);
    }
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
    if ((e = launch(fn, dim3((unsigned)ctas), kThreads, Plan<HD, RP>::kBytes, s, args)) != cudaSuccess || p.whole) return e;
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
    *out_bytes = Work(sms, split::tile_rows(n_heads / n_kv_heads, max_new), head_dim).bytes;
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
    const int group = n_heads / n_kv_heads, rp = split::tile_rows(group, max_new), tokens = rp / group;
    // every unit has to fit int32, whatever the lengths on the device
    const int64_t pairs = ((int64_t)nseq + rows / tokens) * n_kv_heads;
    if (pairs > 0x7fffffffll / ((table_pages + 1) / 2))
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
    p.tokens = tokens;
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
        e = rp == 16 ? run8<128, 16>(p, sms, s) : rp == 32 ? run8<128, 32>(p, sms, s) : rp == 64 ? run8<128, 64>(p, sms, s)
                                                                                            : run8<128, 128>(p, sms, s);
    else
        e = rp == 16 ? run8<64, 16>(p, sms, s) : rp == 32 ? run8<64, 32>(p, sms, s) : rp == 64 ? run8<64, 64>(p, sms, s)
                                                                                          : run8<64, 128>(p, sms, s);
    return e == cudaSuccess ? SPEC_OK : failed(e);
}

}  // extern "C"
