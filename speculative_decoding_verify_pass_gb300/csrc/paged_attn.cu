// Attention of each sequence's newest positions over a paged cache, on the
// fifth-generation tensor cores (tcgen05, accumulators in tensor memory).
//
// For a kv head, R = tokens * G query rows (G query heads per kv head) meet
// every key, so keys and head dimensions run along the 128 tensor-memory lanes
// and the rows are the narrow side.  Per 128-position chunk (two pages):
//     S^T = K Q^T      M = 128 keys,       N = R rounded up to 16, K = head dim
//     P^T = exp2(scale log2e S^T - m)
//     O^T += V^T P^T   M = head dimensions, N as above,            K = 128 keys
// TMA tiles of 64 positions x 64 dimensions land with the 128-byte swizzle and
// are MMA operands as they lie: K rows are K-major, V rows are MN-major (V^T
// without a transpose).  P^T is kept as a bf16 high and a bf16 low part (about
// 16 significant bits), so that only the result's own rounding shows.
//
// The softmax needs no maximum of its own per chunk: m is a reference that
// every row takes from its segment's first chunk.  A later score may exceed it
// by up to 2^40 (fp32 and bf16 hold that), and only if one exceeds it by more do
// the row's reference, sum and O^T get rescaled.  So per chunk and element there
// is one multiply-add, one exp2, one add to the thread's own partial sum and the
// two roundings; nothing crosses lanes until the segment ends.
//
// Roles: warps 0-7 softmax (thread = key, then head dimension; each warpgroup
// half of the rows), warp 8 issues the MMAs, warp 9 the TMA copies.  S^T of the
// next chunk is computed while a chunk's softmax runs.  One CTA per SM, each
// with the same number of chunks (paged_split.h); a second kernel joins the
// pairs that were split between CTAs.
#include <cuda.h>
#include <math.h>

#include "internal.h"
#include "paged_split.h"
#include "spec.h"

namespace sv {
namespace {

using split::kChunk;

constexpr int kSoftWarps = 8;
constexpr int kMmaWarp = kSoftWarps, kLoadWarp = kSoftWarps + 1;
constexpr int kThreads = 32 * (kSoftWarps + 2);
constexpr float kLimit = 40.f;          // log2 by which a score may exceed its row's reference
constexpr float kNone = -1e30f;         // reference of a row that has seen no key

// What the join kernel needs to know of the pair that begins in a CTA and goes on in the next ones.
struct Meta {
    int count;                  // partials (0: no such pair)
    int slot;                   // the owner's slot
    int rows;                   // R
    int head;                   // first query head
    int row0;                   // first row of the call
    int last0;                  // last visible position of the first token
    int pad[2];
};

struct PagedParams {
    CUtensorMap mq, mk, mv;
    const int *row_start, *len, *tables;
    int table_pages, nseq, rows, hq, hkv, group, tokens;
    float scale_log2;
    const uint16_t* vpool;
    int num_pages;
    uint16_t* out;
    long long out_stride;
    int* err;
    float* part_o;              // [2 * ctas][RP][HD]
    float2* part_ml;            // [2 * ctas][RP] (reference, sum)
    Meta* meta;                 // [ctas]
};

// Shared-memory plan: NQ query tiles, NP pairs of P^T parts, NS slots that
// alternately take a chunk's K and V.
template <int HD, int RP>
struct Plan {
    static constexpr int kSlot = kChunk * HD * 2;
    static constexpr int kQ = RP * HD * 2;
    static constexpr int kP = kChunk * RP * 2;              // one part
    static constexpr int NQ = RP <= 32 ? 2 : 1;
    static constexpr int NP = RP <= 64 ? 2 : 1;
    static constexpr int kFixed = NQ * kQ + NP * 2 * kP + 2048;   // alignment, pad after the last slot
    static constexpr int kMost = 227 * 1024 - (6144 + 40 * RP) - kFixed; // less the static arrays
    static constexpr int NS = kMost / kSlot < 8 ? kMost / kSlot : 8;
    static constexpr int kBytes = kFixed + NS * kSlot;
    static constexpr int kCols = 4 * RP;                    // tensor-memory columns: S^T x 2, O^T x 2
    static_assert(NS >= 3, "a chunk's K and the previous chunk's V are live together");
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

// N consecutive fp32 columns of this warp's 32 lanes (N = 8, 16, 32).
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t t, float* v);
template <>
__device__ __forceinline__ void tmem_ld<8>(uint32_t t, float* v) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(t)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st8(uint32_t t, const float* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
                 "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
                 "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two floats rounded to nearest even, a in the low half.
__device__ __forceinline__ uint32_t cvt_bf16x2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// True in every one of n threads of barrier id when any of them says so.
__device__ __forceinline__ bool bar_any(int id, int n, bool any) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(n), "r"((uint32_t)any)
        : "memory");
    return r != 0;
}

// Bounded wait; a wait that gives up raises `dead`, which ends every later one.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* dead) {
    for (uint32_t i = 0; i < (1u << 22); ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (i > 256) __nanosleep(i < 4096 ? 32 : 256);
        if ((i & 255) == 255 && *dead) return false;
    }
    *dead = 1;
    return false;
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* dead) {
    return mbar_try_wait(bar, parity) || wait_slow(bar, parity, dead);
}
// After a failed wait: let what is in flight finish before the CTA ends.
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
    for (uint32_t i = 0; i < (1u << 20) && !mbar_try_wait(bar, parity); ++i) __nanosleep(64);
}

// A CTA's segments in order; every role walks its own copy.
struct Walk {
    const PagedParams& p;
    const int* first;           // [nseq + 1] in shared memory
    int u, end;                 // next unit, end of the CTA's range
    int q = -1, q0 = 0, q1 = 0; // sequence and its units
    int rows = 0, len = 0, row_base = 0, chunks = 1;
    // the segment
    int head = 0, block = 0, c0 = 0, c1 = 0, R = 0, seg = -1;

    __device__ Walk(const PagedParams& pp, const int* f, int begin, int e) : p(pp), first(f), u(begin), end(e) {}
    __device__ __forceinline__ bool next() {
        if (u >= end) return false;
        if (q < 0 || u >= q1) {
            q = split::sequence_of(first, p.nseq, u);
            q0 = first[q];
            q1 = first[q + 1];
            row_base = p.row_start[q];
            rows = p.row_start[q + 1] - row_base;
            len = p.len[q];
            chunks = split::chunks_of(len);
        }
        const int pair = (u - q0) / chunks;
        block = pair / p.hkv;
        head = pair - block * p.hkv;
        c0 = u - q0 - pair * chunks;
        c1 = min(chunks, c0 + end - u);
        R = min(p.tokens, rows - block * p.tokens) * p.group;
        u += c1 - c0;
        ++seg;
        return true;
    }
    __device__ __forceinline__ bool whole() const { return c0 == 0 && c1 == chunks; }
    // last position that the block's first token sees
    __device__ __forceinline__ int last0() const { return len - rows + block * p.tokens; }
};

template <int HD, int RP>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_kernel(const __grid_constant__ PagedParams p) {
    using L = Plan<HD, RP>;
    constexpr int NS = L::NS, NP = L::NP, NQ = L::NQ;
    constexpr int CW = RP / 2;          // rows of a warpgroup
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t kv_full[NS], kv_empty[NS], q_full[NQ], q_empty[NQ], s_full[2], s_empty[2], p_full[NP], p_empty[NP],
        o_full[2], o_empty[2], fin;
    __shared__ uint32_t tmem_base;
    __shared__ int dead, poison[2], total;
    __shared__ int first[split::kMaxSeqs + 1];
    __shared__ long long warp_sum[kThreads / 32];
    __shared__ __align__(16) float mref[RP];            // reference of each row
    __shared__ __align__(16) float xred[4][RP];         // per lane quadrant: maxima, then sums
    __shared__ __align__(16) int tok[RP];               // token of each row
    __shared__ long long col_off[RP];                   // its offset in the output

    uint8_t* base = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* slots = base;
    uint8_t* qs = slots + NS * L::kSlot + 1024;         // 1 KB: an M = 128 MMA over 64 dimensions reads past its slot
    uint8_t* ps = qs + NQ * L::kQ;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 1);
        }
        for (int i = 0; i < NQ; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], kSoftWarps);
            mbar_init(&o_full[i], 1);
            mbar_init(&o_empty[i], kSoftWarps);
            poison[i] = 0;
        }
        for (int i = 0; i < NP; ++i) {
            mbar_init(&p_full[i], kSoftWarps);
            mbar_init(&p_empty[i], 1);
        }
        mbar_init(&fin, 1);
        fence_barrier_init();
        dead = 0;
        first[0] = 0;
    }
    for (int i = tid; i < RP; i += kThreads) {
        const int t = i / p.group;
        tok[i] = t;
        col_off[i] = t * p.out_stride + (long long)(i - t * p.group) * HD;
    }
    if (warp == kMmaWarp) tmem_alloc(&tmem_base, L::kCols);
    pdl_wait();
    pdl_launch_dependents();

    // first[q]: exclusive sums of the sequences' units, 4 sequences a thread
    {
        long long v[4], sum = 0;   // 64 bits: row ranges that overlap can pass any bound
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int q = tid * 4 + k;
            v[k] = 0;
            if (q < p.nseq) {
                const int r0 = p.row_start[q], r1 = p.row_start[q + 1], n = p.len[q];
                const bool bad_rows = r0 < 0 || r1 < r0 || r1 > p.rows;
                const bool bad_len = n < 0 || n > (long long)p.table_pages * SPEC_PAGE;
                if (bad_rows || bad_len) {
                    if (blockIdx.x == 0 && p.err) atomicCAS(p.err, 0, bad_rows ? SPEC_PAGED_BAD_ROWS : SPEC_PAGED_BAD_LENGTH);
                } else {
                    v[k] = split::units_of(r1 - r0, n, p.tokens, p.hkv);
                }
            }
            sum += v[k];
        }
        long long inc = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        if (lane == 31) warp_sum[warp] = inc;
        __syncthreads();
        long long run = inc - sum;
        for (int w = 0; w < warp; ++w) run += warp_sum[w];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            run += v[k];
            if (tid * 4 + k < p.nseq) first[tid * 4 + k + 1] = (int)run;
        }
        if (tid == kThreads - 1) {
            total = run > 0x7fffffff ? 0 : (int)run;
            if (run > 0x7fffffff && blockIdx.x == 0 && p.err) atomicCAS(p.err, 0, SPEC_PAGED_BAD_ROWS);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    const int T = total, work = split::working(gridDim.x, T);
    const int begin = split::begin_of(blockIdx.x, T, work), end = split::begin_of(blockIdx.x + 1, T, work);
    volatile int* deadp = &dead;

    if (warp == kLoadWarp) {
        // ---------------- TMA copies (lane 0 issues; the lanes look up pages) ----------------
        Walk w(p, first, begin, end);
        int fill = 0;
        bool ok = true;
        while (ok && w.next()) {
            if (lane == 0) {
                uint64_t* qf = &q_full[w.seg % NQ];
                ok = wait(&q_empty[w.seg % NQ], ((w.seg / NQ) & 1) ^ 1, deadp);
                if (ok) {
                    mbar_arrive_expect_tx(qf, (uint32_t)(p.tokens * p.group * HD * 2));
#pragma unroll
                    for (int hf = 0; hf < HD / 64; ++hf)
                        tma3(qs + (w.seg % NQ) * L::kQ + hf * RP * 128, &p.mq, hf * 64, w.head * p.group,
                             w.row_base + w.block * p.tokens, qf);
                }
            }
            const int held = (w.len + SPEC_PAGE - 1) / SPEC_PAGE;
            const int* tab = p.tables + (size_t)w.q * p.table_pages;
            int z0 = -1, z1 = -1;               // the lane's chunk: tensor-map rows of its two pages
            for (int c = w.c0; c < w.c1; ++c) {
                const int k = (c - w.c0) & 31;
                if (k == 0) {                   // the next 32 chunks' pages, one chunk a lane
                    const int e = 2 * (c + lane);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        int z = -1;
                        if (c + lane < w.c1 && e + i < held) {
                            const int page = tab[e + i];
                            if (page >= 0 && page < p.num_pages) z = page * p.hkv + w.head;
                            else if (p.err) atomicCAS(p.err, 0, SPEC_PAGED_BAD_PAGE);
                        }
                        if (i) z1 = z;
                        else z0 = z;
                    }
                }
                const int a0 = __shfl_sync(0xffffffffu, z0, k), a1 = __shfl_sync(0xffffffffu, z1, k);
                if (lane == 0 && ok) {
                    const int n = min(2, held - 2 * c);   // pages that exist (a bad one reads as zeros: z = -1)
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const int s = fill % NS;
                        ok = ok && wait(&kv_empty[s], ((fill / NS) & 1) ^ 1, deadp);
                        if (!ok) break;
                        uint8_t* dst = slots + s * L::kSlot;
                        const CUtensorMap* map = kv ? &p.mv : &p.mk;
                        mbar_arrive_expect_tx(&kv_full[s], n > 0 ? (uint32_t)(n * SPEC_PAGE * HD * 2) : 0u);
#pragma unroll
                        for (int hf = 0; hf < HD / 64; ++hf) {
                            if (n > 0) tma3(dst + hf * kChunk * 128, map, hf * 64, 0, a0, &kv_full[s]);
                            if (n > 1) tma3(dst + hf * kChunk * 128 + SPEC_PAGE * 128, map, hf * 64, 0, a1, &kv_full[s]);
                        }
                        ++fill;
                    }
                }
            }
            ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
        }
        if (lane == 0 && *deadp) {
            for (int f = fill > NS ? fill - NS : 0; f < fill; ++f) drain(&kv_full[f % NS], (f / NS) & 1);
            for (int s = w.seg - NQ + 1 < 0 ? 0 : w.seg - NQ + 1; s <= w.seg; ++s) drain(&q_full[s % NQ], (s / NQ) & 1);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ---------------- MMAs (one thread): S^T one unit ahead of O^T ----------------
        if (lane == 0) {
            Walk ws(p, first, begin, end), wo(p, first, begin, end);
            const uint32_t sa = smem_u32(slots), qa = smem_u32(qs), pa = smem_u32(ps);
            bool ok = true;
            int cs = 0, co = 0;                 // next chunk of ws' and wo's segments
            const int n = end - begin;
            for (int i = 0; i <= n && ok; ++i) {
                if (i < n) {                    // S^T of unit i
                    const bool head = i == 0 || cs == ws.c1;
                    if (head) {
                        ws.next();
                        cs = ws.c0;
                        ok = ok && wait(&q_full[ws.seg % NQ], (ws.seg / NQ) & 1, deadp);
                    }
                    const int f = 2 * i, s = f % NS;
                    ok = ok && wait(&kv_full[s], (f / NS) & 1, deadp);
                    ok = ok && wait(&s_empty[i & 1], ((i >> 1) & 1) ^ 1, deadp);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t id = umma_idesc_bf16(128, (ws.R + 15) & ~15);
                    const uint64_t dk = desc_sw128(sa + s * L::kSlot, 16, 1024);
                    const uint64_t dq = desc_sw128(qa + (ws.seg % NQ) * L::kQ, 16, 1024);
#pragma unroll
                    for (int k = 0; k < HD / 16; ++k)
                        umma_bf16_id(tmem + (i & 1) * RP, dk + (k >> 2) * (kChunk * 128 >> 4) + (k & 3) * 2,
                                     dq + (k >> 2) * (RP * 128 >> 4) + (k & 3) * 2, id, k > 0);
                    umma_commit(&s_full[i & 1]);
                    umma_commit(&kv_empty[s]);
                    if (++cs == ws.c1) umma_commit(&q_empty[ws.seg % NQ]);
                }
                if (i > 0) {                    // O^T of unit i - 1
                    const int j = i - 1;
                    if (j == 0 || co == wo.c1) {
                        wo.next();
                        co = wo.c0;
                        ok = ok && wait(&o_empty[wo.seg & 1], ((wo.seg >> 1) & 1) ^ 1, deadp);
                    }
                    const int f = 2 * j + 1, s = f % NS;
                    ok = ok && wait(&kv_full[s], (f / NS) & 1, deadp);
                    ok = ok && wait(&p_full[j % NP], (j / NP) & 1, deadp);
                    if (!ok) break;
                    tc_fence_after();
                    // A = V^T and B = P^T, both MN-major
                    const uint32_t id = umma_idesc_bf16(128, (wo.R + 15) & ~15) | (1u << 15) | (1u << 16);
                    const uint64_t dv = desc_sw128(sa + s * L::kSlot, HD == 128 ? kChunk * 128 : 1024, 1024);
                    const uint64_t dp = umma_desc_kmajor(pa + (j % NP) * 2 * L::kP, 128, kChunk * 16);
                    const uint32_t o = tmem + 2 * RP + (wo.seg & 1) * RP;
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int k = 0; k < kChunk / 16; ++k)
                            umma_bf16_id(o, dv + k * (2048 >> 4), dp + part * (L::kP >> 4) + k * (256 >> 4), id,
                                         co != wo.c0 || (part | k) != 0);
                    umma_commit(&kv_empty[s]);
                    umma_commit(&p_empty[j % NP]);
                    if (++co == wo.c1) umma_commit(&o_full[wo.seg & 1]);
                }
            }
            if (!ok) {
                umma_commit(&fin);
                drain(&fin, 0);
            }
        }
        __syncwarp();
    } else {
        // ---------------- softmax and results: thread = key, then head dimension ----------------
        const int wg = warp >> 2, qd = warp & 3;
        const uint32_t lanes = (uint32_t)(qd * 32) << 16;
        const int key = qd * 32 + lane;
        const int col0 = wg * CW;               // the warpgroup's first row
        const int bar = 1 + wg;
        Walk w(p, first, begin, end);
        int i = 0;                              // unit
        bool ok = true;
        while (w.next()) {
            const int last0 = w.last0(), last_max = last0 + tok[w.R - 1];
            const bool idle = w.R <= col0;
            float l[CW];
#pragma unroll
            for (int j = 0; j < CW; ++j) l[j] = 0.f;
            if (tid == 0) poison[w.seg & 1] = 0;
            for (int c = w.c0; c < w.c1; ++c, ++i) {
                const int kp = c * kChunk + key;
                ok = ok && wait(&s_full[i & 1], (i >> 1) & 1, deadp);
                tc_fence_after();
                float s[CW];
                if (!idle) {
#pragma unroll
                    for (int j = 0; j < CW; j += 8) tmem_ld<8>(tmem + lanes + (i & 1) * RP + col0 + j, s + j);
                    tmem_wait_ld();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_empty[i & 1]);
                const bool masked = (c + 1) * kChunk - 1 > last0;   // some row does not see all of the chunk
                if (!idle) {
                    if (masked) {
#pragma unroll
                        for (int j = 0; j < CW; ++j)
                            if (kp > last0 + tok[col0 + j]) s[j] = -INFINITY;
                    }
                    float top = kNone;
                    if (c != w.c0) {
#pragma unroll
                        for (int j = 0; j < CW; j += 4) {
                            const float4 m = *reinterpret_cast<const float4*>(&mref[col0 + j]);
                            top = fmaxf(top, fmaxf(fmaxf(fmaf(s[j], p.scale_log2, -m.x), fmaf(s[j + 1], p.scale_log2, -m.y)),
                                                   fmaxf(fmaf(s[j + 2], p.scale_log2, -m.z), fmaf(s[j + 3], p.scale_log2, -m.w))));
                        }
                    }
                    if (bar_any(bar, 128, c == w.c0 || top > kLimit)) {
                        // new references: the chunk's row maxima over the four quadrants
#pragma unroll
                        for (int j = 0; j < CW; ++j) {
                            const float m = warp_max_exact(s[j]);
                            if (lane == 0) xred[qd][col0 + j] = m;
                        }
                        named_bar_sync(bar, 128);
                        if (c != w.c0) {        // O^T holds the chunks before: rescale it with the sums
                            ok = ok && wait(&p_empty[(i - 1) % NP], ((i - 1) / NP) & 1, deadp);
                            tc_fence_after();
                        }
#pragma unroll
                        for (int j = 0; j < CW; j += 8) {
                            float o[8] = {};
                            const uint32_t at = tmem + lanes + 2 * RP + (w.seg & 1) * RP + col0 + j;
                            if (c != w.c0) {
                                tmem_ld<8>(at, o);
                                tmem_wait_ld();
                            }
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const int r = col0 + j + e;
                                const float m = fmaxf(fmaxf(xred[0][r], xred[1][r]), fmaxf(xred[2][r], xred[3][r])) * p.scale_log2;
                                const float old = c != w.c0 ? mref[r] : kNone;
                                const float f = ex2_approx(old - fmaxf(old, m));
                                l[j + e] *= f;
                                o[e] *= f;
                            }
                            if (c != w.c0) tmem_st8(at, o);
                        }
                        if (c != w.c0) {
                            tmem_wait_st();
                            tc_fence_before();
                        }
                        named_bar_sync(bar, 128);   // everyone has read the old references
                        for (int r = col0 + key; r < col0 + CW; r += 128) {
                            const float m = fmaxf(fmaxf(xred[0][r], xred[1][r]), fmaxf(xred[2][r], xred[3][r])) * p.scale_log2;
                            const float old = c != w.c0 ? mref[r] : kNone;
                            mref[r] = r >= w.R ? INFINITY : fmaxf(old, m);   // rows past R weigh nothing
                        }
                        named_bar_sync(bar, 128);
                    }
#pragma unroll
                    for (int j = 0; j < CW; j += 4) {
                        const float4 m = *reinterpret_cast<const float4*>(&mref[col0 + j]);
                        s[j] = ex2_approx(fmaf(s[j], p.scale_log2, -m.x));
                        s[j + 1] = ex2_approx(fmaf(s[j + 1], p.scale_log2, -m.y));
                        s[j + 2] = ex2_approx(fmaf(s[j + 2], p.scale_log2, -m.z));
                        s[j + 3] = ex2_approx(fmaf(s[j + 3], p.scale_log2, -m.w));
#pragma unroll
                        for (int e = 0; e < 4; ++e) l[j + e] += s[j + e];
                    }
                }
                if (i >= NP) ok = ok && wait(&p_empty[i % NP], ((i / NP) & 1) ^ 1, deadp);
                if (!idle) {
                    uint8_t* ph = ps + (i % NP) * 2 * L::kP + key * 16;
#pragma unroll
                    for (int j = 0; j < CW; j += 8) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float a = s[j + 2 * e], b = s[j + 2 * e + 1];
                            hi[e] = cvt_bf16x2(a, b);
                            lo[e] = cvt_bf16x2(a - __uint_as_float(hi[e] << 16), b - __uint_as_float(hi[e] & 0xFFFF0000u));
                        }
                        uint8_t* dst = ph + ((col0 + j) >> 3) * (kChunk * 16);
                        *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(dst + L::kP) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                }
                if (masked && wg == 0) {
                    // Values of positions that some row does not see: behind the
                    // length they become zero (a weight of zero does not silence a
                    // NaN), between the rows' last positions non-finite ones do,
                    // and are added at the end to the rows that see them.
                    const int f = 2 * i + 1, sl = f % NS;
                    ok = ok && wait(&kv_full[sl], (f / NS) & 1, deadp);
                    uint8_t* v = slots + sl * L::kSlot;
                    const int from = max(0, last0 + 1 - c * kChunk), live = w.len - c * kChunk;
                    for (int t = from * (HD / 8) + key; t < kChunk * (HD / 8); t += 128) {
                        const int r = t / (HD / 8), d8 = t % (HD / 8);
                        uint4* at = reinterpret_cast<uint4*>(v + (d8 >> 3) * kChunk * 128 + r * 128 + (((d8 & 7) ^ (r & 7)) << 4));
                        if (r >= live) {
                            *at = make_uint4(0u, 0u, 0u, 0u);
                        } else {
                            uint4 x = *at;
                            uint32_t* e = &x.x;
                            bool hit = false;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if ((e[k] & 0x7F80u) == 0x7F80u) hit = true, e[k] &= 0xFFFF0000u;
                                if ((e[k] & 0x7F800000u) == 0x7F800000u) hit = true, e[k] &= 0xFFFFu;
                            }
                            if (hit) {
                                *at = x;
                                poison[w.seg & 1] = 1;
                            }
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[i % NP]);
            }
            // ---- the segment's rows ----
            const bool whole = w.whole();
            const int slot = 2 * blockIdx.x + (w.u - (w.c1 - w.c0) == begin ? 0 : 1);
            if (!idle) {
#pragma unroll
                for (int j = 0; j < CW; ++j) {
                    float x = l[j];
#pragma unroll
                    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
                    if (lane == 0) xred[qd][col0 + j] = x;
                }
                named_bar_sync(bar, 128);
            }
            ok = ok && wait(&o_full[w.seg & 1], (w.seg >> 1) & 1, deadp);
            tc_fence_after();
            if (!idle) {
                const int d = key;
                const bool bad = poison[w.seg & 1] != 0;
                uint16_t* out = p.out + (long long)(w.row_base + w.block * p.tokens) * p.out_stride +
                                (long long)w.head * p.group * HD + d;
                if (!whole)
                    for (int r = col0 + key; r < min(w.R, col0 + CW); r += 128)
                        p.part_ml[(size_t)slot * RP + r] =
                            make_float2(mref[r], xred[0][r] + xred[1][r] + xred[2][r] + xred[3][r]);
#pragma unroll 1
                for (int j = 0; j < CW && col0 + j < w.R; j += 8) {
                    float o[8];
                    tmem_ld<8>(tmem + lanes + 2 * RP + (w.seg & 1) * RP + col0 + j, o);
                    tmem_wait_ld();
                    if (d < HD) {
                        if (bad)
                            for (int t = max(last0 + 1, w.c0 * kChunk); t <= min(last_max, w.c1 * kChunk - 1); ++t) {
                                const int page = p.tables[(size_t)w.q * p.table_pages + t / SPEC_PAGE];
                                if (page < 0 || page >= p.num_pages) continue;
                                const float v = bf2f(p.vpool[(((size_t)page * p.hkv + w.head) * SPEC_PAGE + t % SPEC_PAGE) * HD + d]);
                                if (!isfinite(v))
#pragma unroll
                                    for (int e = 0; e < 8; ++e)
                                        if (t <= last0 + tok[col0 + j + e]) o[e] += v;
                            }
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int r = col0 + j + e;
                            if (r < w.R) {
                                if (whole) {
                                    const float sum = xred[0][r] + xred[1][r] + xred[2][r] + xred[3][r];
                                    out[col_off[r]] = f2bf(last0 + tok[r] >= 0 ? o[e] / sum : 0.f);
                                } else {
                                    p.part_o[((size_t)slot * RP + r) * HD + d] = o[e];
                                }
                            }
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_empty[w.seg & 1]);
        }
        // what the join kernel has to do for the pair that begins here and goes on
        if (tid == 0) {
            Meta m = {};
            if (w.seg >= 0 && w.c1 < w.chunks) {
                const int pair_begin = w.u - w.c1;           // unit of the pair's chunk 0
                if (pair_begin >= begin) {
                    m.count = split::contributors(blockIdx.x, pair_begin + w.chunks, T, work);
                    m.slot = 2 * blockIdx.x + (pair_begin == begin ? 0 : 1);
                    m.rows = w.R;
                    m.head = w.head * p.group;
                    m.row0 = w.row_base + w.block * p.tokens;
                    m.last0 = w.last0();
                }
            }
            p.meta[blockIdx.x] = m;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && dead && p.err) atomicCAS(p.err, 0, SPEC_PAGED_TIMEOUT);
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kCols);
    }
}

// Joins the partials of each pair that CTAs shared: CTA (c, y) takes rows 8y,
// 8y + 8 gridDim.y, .. of the pair that begins in CTA c, one warp a row.
template <int HD>
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ PagedParams p, int rp) {
    pdl_wait();
    pdl_launch_dependents();
    const Meta m = p.meta[blockIdx.x];
    const int lane = threadIdx.x & 31;
    constexpr int V = HD / 32;
    for (int r = blockIdx.y * 8 + (threadIdx.x >> 5); r < m.rows && m.count > 0; r += gridDim.y * 8) {
        // partial t of the pair: the owner's slot, then the first slots of the CTAs after it
        auto at = [&](int t) { return (size_t)(t ? 2 * (blockIdx.x + t) : m.slot) * rp + r; };
        float M = kNone;
        for (int t = lane; t < m.count; t += 32) M = fmaxf(M, p.part_ml[at(t)].x);
#pragma unroll
        for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
        float sum = 0.f, o[V] = {};
#pragma unroll 8
        for (int t = 0; t < m.count; ++t) {
            const float2 ml = p.part_ml[at(t)];
            const float* src = p.part_o + at(t) * HD + lane * V;
            const float f = ex2_approx(ml.x - M);
            sum += f * ml.y;
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] += f * src[e];
        }
        const int t = r / p.group;
        uint16_t* out = p.out + (long long)(m.row0 + t) * p.out_stride + (long long)(m.head + r - t * p.group) * HD + lane * V;
#pragma unroll
        for (int e = 0; e < V; ++e) out[e] = f2bf(m.last0 + t >= 0 ? o[e] / sum : 0.f);
    }
}

spec_status bad(const char* msg) {
    set_last_error(msg);
    return SPEC_ERR_INVALID_ARG;
}

spec_status failed(cudaError_t e) {
    set_last_error(cudaGetErrorString(e));
    return SPEC_ERR_CUDA;
}

bool misaligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// What the head layout has to satisfy; null when it does.
const char* head_error(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t max_new) {
    if (head_dim != 64 && head_dim != 128) return "spec_paged_attention: head_dim must be 64 or 128";
    if (n_kv_heads < 1 || n_kv_heads > 1024 || n_heads < n_kv_heads || n_heads % n_kv_heads)
        return "spec_paged_attention: n_heads must be a multiple of n_kv_heads, 1..1024";
    if (n_heads / n_kv_heads > 128) return "spec_paged_attention: at most 128 query heads per kv head";
    if (max_new < 1) return "spec_paged_attention: max_new must be at least 1";
    return nullptr;
}

// Workspace: partial outputs, (reference, sum) pairs, one Meta per CTA.
struct Work {
    size_t o, ml, meta, bytes;
    Work(int ctas, int rp, int hd) {
        o = 0;
        ml = (size_t)2 * ctas * rp * hd * 4;
        meta = ml + (size_t)2 * ctas * rp * 8;
        bytes = (meta + (size_t)ctas * sizeof(Meta) + 255) & ~(size_t)255;
    }
};

// SMs of the current device, its index checked; 0 on an error.
int current_sms() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return sms;
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
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

cudaError_t launch(const void* fn, dim3 grid, unsigned block, size_t smem, cudaStream_t s, void** args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

template <int HD, int RP>
cudaError_t run(PagedParams& p, int ctas, cudaStream_t s) {
    const void* fn = (const void*)paged_attn_kernel<HD, RP>;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Plan<HD, RP>::kBytes);
    if (e != cudaSuccess) return e;
    void* args[] = {&p};
    if ((e = launch(fn, dim3((unsigned)ctas), kThreads, Plan<HD, RP>::kBytes, s, args)) != cudaSuccess) return e;
    int rp = RP;
    void* jargs[] = {&p, &rp};
    return launch((const void*)paged_join_kernel<HD>, dim3((unsigned)ctas, RP / 16), 256, 0, s, jargs);
}

}  // namespace
}  // namespace sv

extern "C" {

using namespace sv;

spec_status spec_paged_attention_workspace(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t max_new,
                                           size_t* out_bytes) {
    if (!out_bytes) return bad("spec_paged_attention_workspace: null pointer");
    if (const char* e = head_error(n_heads, n_kv_heads, head_dim, max_new)) return bad(e);
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
    if (!d_q || !d_row_start || !d_len || !d_tables || !d_kpool || !d_vpool || !d_out || !d_work)
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
    if (work_bytes < Work(1, rp, head_dim).bytes) return bad("spec_paged_attention: work_bytes is less than these heads need");
    const int sms = current_sms();
    if (!sms) {
        set_last_error("spec_paged_attention: no current CUDA device");
        return SPEC_ERR_CUDA;
    }
    const Work work(sms, rp, head_dim);
    if (work_bytes < work.bytes) return bad("spec_paged_attention: work_bytes is less than these heads need");
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
    p.hq = n_heads;
    p.hkv = n_kv_heads;
    p.group = group;
    p.tokens = tokens;
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
