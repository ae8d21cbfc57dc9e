// What the attention kernels over a paged cache share, whatever its pages hold:
// tensor-memory helpers, the walk over a segment's pages, the join of pairs that CTAs
// shared, and the host's part of a launch.
#pragma once

#include <cuda.h>
#include <float.h>
#include <math.h>

#include "internal.h"
#include "paged_split.h"
#include "spec.h"

namespace sv {
namespace {

using split::kChunk;

constexpr float kNone = -FLT_MAX;       // reference of a row that has seen no key: no score lies below it

// A split pair, as the join kernel sees it from one of its CTAs.
struct Meta {
    int count;                  // partials (0: no such pair)
    int owner;                  // the CTA where it begins
    int slot;                   // the owner's slot
    int rows;                   // R
    int head;                   // first query head
    int row0;                   // first row of the call
    int last0;                  // last visible position of the first token
    int skip;                   // query heads of the first token in front of the first row
};

// What a call is about, apart from the tensor maps of its operands.
struct PagedCommon {
    const int *row_start, *len, *tables;
    int table_pages, nseq, rows, hkv, group, tokens;
    int whole;                  // pairs are not split: a CTA takes those that begin in its range
    float scale_log2;
    int num_pages;
    uint16_t* out;
    long long out_stride;
    int* err;
    float* part_o;              // [2 * ctas][RP][HD]
    float2* part_ml;            // [2 * ctas][RP] (reference, sum)
    Meta* meta;                 // [ctas][2]: the pair that goes on into the CTA, the pair that begins in it and goes on
};

// 8 or 16 consecutive fp32 columns of this warp's 32 lanes, not waited for.
__device__ __forceinline__ void tmem_ld8_async(uint32_t t, float* v) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(t)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld16_async(uint32_t t, float* v) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
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

// Two fp32 operations in one instruction.
struct F2 {
    uint64_t v;
    __device__ __forceinline__ F2() {}
    __device__ __forceinline__ F2(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ void get(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
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

// True in one lane of a converged warp, always the same one.  Issuing MMAs and
// copies under this predicate (and not under lane == 0) tells the compiler that
// one thread issues them; otherwise every issue pays for finding that out.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// The SM's clock: waits are bounded in time, by 2^31 cycles (about a second).
__device__ __forceinline__ uint32_t cycles() {
    uint32_t c;
    asm volatile("mov.u32 %0, %%clock;" : "=r"(c));
    return c;
}

// Position in a ring of N buffers: index and the parity of its current round.
template <int N>
struct Ring {
    int at = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void step() {
        if (++at == N) at = 0, round ^= 1;
    }
};

// The pages of a segment's chunks, looked up 32 chunks at a time, one a lane.
struct PageWalk {
    int y0 = -1, y1 = -1;       // the lane's chunk: tensor-map rows of its two pages
    int z0 = -1, z1 = -1;       // the current chunk's (a bad page's -1 lies outside the pool and reads as zeros)
    int count = 0;              // and how many of them exist
    template <class Seg>
    __device__ __forceinline__ void at(const PagedCommon& p, const Seg& s, int k, int lane) {
        const int held = (s.len + SPEC_PAGE - 1) / SPEC_PAGE, c = s.c0 + k;
        if ((k & 31) == 0) {
            const int* tab = p.tables + (size_t)s.q * p.table_pages + 2 * (c + lane);
            const int have = k + lane < s.units ? held - 2 * (c + lane) : 0;
            const int a = have > 0 ? tab[0] : -1, b = have > 1 ? tab[1] : -1;
            const bool oka = a >= 0 && a < p.num_pages, okb = b >= 0 && b < p.num_pages;
            if (p.err && ((have > 0 && !oka) || (have > 1 && !okb))) atomicCAS(p.err, 0, SPEC_PAGED_BAD_PAGE);
            y0 = oka ? a * p.hkv + s.head : -1;
            y1 = okb ? b * p.hkv + s.head : -1;
        }
        z0 = __shfl_sync(0xffffffffu, y0, k & 31);
        z1 = __shfl_sync(0xffffffffu, y1, k & 31);
        count = max(0, min(2, held - 2 * c));
    }
};

template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Joins the partials of each pair that CTAs shared: CTA (c, y) works for the pair
// that goes on into attention CTA c (y even) or begins in it and goes on (odd).
// The CTAs of a pair deal its rows among themselves (t of n takes rows t, t + n,
// ..): the more partials a row has, the more CTAs read them.  Up to 8 partials a warp joins a row, its
// loads all in flight at once; above, the CTA's 8 warps share the row's partials.
constexpr int kJoinFew = 8, kJoinWarps = 8;

template <int HD>
__global__ void __launch_bounds__(32 * kJoinWarps) paged_join_kernel(const __grid_constant__ PagedCommon p, int rp) {
    constexpr int V = HD / 32;
    __shared__ float so[kJoinWarps][HD];
    __shared__ float ssum[kJoinWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_launch_dependents();
    {
        const Meta m = p.meta[2 * blockIdx.x + (blockIdx.y & 1)];
        if (m.count == 0) return;
        const int mine = blockIdx.x - m.owner, y0 = blockIdx.y >> 1, ny = gridDim.y >> 1;
        // partial t of the pair: the owner's slot, then the first slots of the CTAs after it
        auto at = [&](int r, int t) { return (size_t)(t ? 2 * (m.owner + t) : m.slot) * rp + r; };
        auto store = [&](int r, const float* o, float sum) {
            const int t = (m.skip + r) / p.group;
            const bool any = m.last0 + t >= 0;
            uint16_t* out = p.out + (long long)(m.row0 + t) * p.out_stride + (long long)(m.head + m.skip + r - t * p.group) * HD + lane * V;
            const float inv = any ? 1.f / sum : 0.f;
            if constexpr (V == 4)
                *reinterpret_cast<uint2*>(out) = any ? make_uint2(cvt_bf16x2(o[0] * inv, o[1] * inv), cvt_bf16x2(o[2] * inv, o[3] * inv))
                                                     : make_uint2(0u, 0u);
            else
                *reinterpret_cast<uint32_t*>(out) = any ? cvt_bf16x2(o[0] * inv, o[1] * inv) : 0u;
        };
        auto load = [&](size_t i, float* v) {
            if constexpr (V == 4) {
                const float4 x = *reinterpret_cast<const float4*>(p.part_o + i * HD + lane * 4);
                v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
            } else {
                const float2 x = *reinterpret_cast<const float2*>(p.part_o + i * HD + lane * 2);
                v[0] = x.x, v[1] = x.y;
            }
        };
        if (m.count <= kJoinFew) {
            for (int r = mine + m.count * (warp + kJoinWarps * y0); r < m.rows; r += m.count * kJoinWarps * ny) {
                float v[kJoinFew][V];
                float2 ml[kJoinFew];
#pragma unroll
                for (int t = 0; t < kJoinFew; ++t)
                    if (t < m.count) {
                        ml[t] = p.part_ml[at(r, t)];
                        load(at(r, t), v[t]);
                    }
                float M = kNone, sum = 0.f, o[V] = {};
#pragma unroll
                for (int t = 0; t < kJoinFew; ++t)
                    if (t < m.count) M = fmaxf(M, ml[t].x);
#pragma unroll
                for (int t = 0; t < kJoinFew; ++t)
                    if (t < m.count) {
                        const float f = ex2_approx(ml[t].x - M);
                        sum += f * ml[t].y;
#pragma unroll
                        for (int e = 0; e < V; ++e) o[e] += f * v[t][e];
                    }
                store(r, o, sum);
            }
        } else {
            for (int r = mine + m.count * y0; r < m.rows; r += m.count * ny) {
                float M = kNone, sum = 0.f, o[V] = {};
                for (int t = lane; t < m.count; t += 32) M = fmaxf(M, p.part_ml[at(r, t)].x);
#pragma unroll
                for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
                for (int t0 = warp; t0 < m.count; t0 += 4 * kJoinWarps) {
                    float v[4][V];
                    float2 ml[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int t = t0 + i * kJoinWarps;
                        if (t < m.count) {
                            ml[i] = p.part_ml[at(r, t)];
                            load(at(r, t), v[i]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (t0 + i * kJoinWarps < m.count) {
                            const float f = ex2_approx(ml[i].x - M);
                            sum += f * ml[i].y;
#pragma unroll
                            for (int e = 0; e < V; ++e) o[e] += f * v[i][e];
                        }
                }
#pragma unroll
                for (int e = 0; e < V; ++e) so[warp][lane * V + e] = o[e];
                if (lane == 0) ssum[warp] = sum;
                __syncthreads();
                if (warp == 0) {
                    sum = 0.f;
#pragma unroll
                    for (int e = 0; e < V; ++e) o[e] = 0.f;
#pragma unroll
                    for (int w = 0; w < kJoinWarps; ++w) {
                        sum += ssum[w];
#pragma unroll
                        for (int e = 0; e < V; ++e) o[e] += so[w][lane * V + e];
                    }
                    store(r, o, sum);
                }
                __syncthreads();
            }
        }
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

// Workspace: partial outputs, (reference, sum) pairs, two Metas per CTA.
struct Work {
    size_t o, ml, meta, bytes;
    Work(int ctas, int rp, int hd) {
        o = 0;
        ml = (size_t)2 * ctas * rp * hd * 4;
        meta = ml + (size_t)2 * ctas * rp * 8;
        bytes = (meta + (size_t)2 * ctas * sizeof(Meta) + 255) & ~(size_t)255;
    }
};

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

}  // namespace
}  // namespace sv
