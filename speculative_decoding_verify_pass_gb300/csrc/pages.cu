// A page pool shared by many sequences: page tables and slot maps stepped on
// the device, and the append of new keys and values at their slots.
//
// One step crops every sequence to `keep` positions and adds `add` new ones
// (the accept/rollback of a verify cycle, DFlash README "Verify" and "Accept",
// and the admission and retirement of sequences, in one call).  With held =
// ceil(len/64) and need = ceil((keep+add)/64), sequence q gives back its table
// entries need..held-1 or takes pages for its entries held..need-1.  In
// (sequence, page) order, three exclusive sums over the sequences number the
// pages given back, the pages taken and the new rows:
//   stack[count + i]          = the i-th page given back
//   the k-th page taken       = stack[count + R - 1 - k]  (R pages given back)
//   slots[row_start[q] + i]   = table[q][(keep+i)/64] * 64 + (keep+i) % 64
// A page on the stack at or above `count` is one given back in this call; it
// is looked up in its old table row, which this call leaves alone, so that no
// thread waits for another's write.
#include <stdio.h>

#include "internal.h"
#include "spec.h"

namespace sv {
namespace {

constexpr int kStepThreads = 1024, kFewThreads = 128;   // one sequence per thread
static_assert(kStepThreads >= SPEC_MAX_SEQS, "one sequence per thread");
constexpr int kPoolTicket = 2;        // header word: CTAs done (0 between launches)

struct StepParams {
    int* pool;
    int num_pages;
    int* tables;
    int table_pages;
    int* len;
    const int* keep;
    const int* add;
    int nseq;
    int* row_start;
    int* slots;
    int row_cap;
};

// Inclusive sums over the CTA's threads (int and 64-bit values at once).
struct Sum3 {
    int rel, alc;
    long long rows;
};
__device__ __forceinline__ Sum3 operator+(const Sum3& a, const Sum3& b) { return {a.rel + b.rel, a.alc + b.alc, a.rows + b.rows}; }
__device__ __forceinline__ Sum3 shfl_up(const Sum3& a, int d) {
    return {__shfl_up_sync(0xffffffffu, a.rel, d), __shfl_up_sync(0xffffffffu, a.alc, d),
            __shfl_up_sync(0xffffffffu, a.rows, d)};
}

// The sequence whose range of the exclusive sums s[0..nseq] holds i: the last
// q with s[q] <= i (its range is not empty when i < s[nseq]).
__device__ __forceinline__ int owner(const int* s, int nseq, int i) {
    int lo = 0, hi = nseq;   // s[lo] <= i < s[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Every CTA forms the same sums; the items (pages given back, pages taken,
// rows) are dealt to all CTAs' threads.  The last CTA to finish (ticket in the
// pool's header, back at zero afterwards) writes the lengths and the header,
// which every CTA has read by then.
template <int T>
__global__ void __launch_bounds__(T) pages_step_kernel(const __grid_constant__ StepParams p) {
    __shared__ int rel[T + 1], alc[T + 1], row[T + 1];
    __shared__ int held[T], need[T], keep[T];
    __shared__ Sum3 part[T / 32];
    __shared__ int last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_launch_dependents();
    int code = 0, newlen = 0;
    Sum3 mine = {0, 0, 0};
    if (tid < p.nseq) {
        const int n = p.len[tid], k = p.keep[tid], a = p.add[tid];
        const long long total = (long long)k + a;
        if (n < 0 || k < 0 || k > n || a < 0 || total > (long long)p.table_pages * SPEC_PAGE ||
            n > (long long)p.table_pages * SPEC_PAGE) {
            code = SPEC_PAGED_BAD_LENGTH;
            held[tid] = need[tid] = keep[tid] = 0;
        } else {
            const int h = (n + SPEC_PAGE - 1) / SPEC_PAGE, d = (int)((total + SPEC_PAGE - 1) / SPEC_PAGE);
            newlen = (int)total;
            held[tid] = h;
            need[tid] = d;
            keep[tid] = k;
            mine = {h > d ? h - d : 0, d > h ? d - h : 0, a};
        }
    }
    Sum3 inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const Sum3 o = shfl_up(inc, d);
        if (lane >= d) inc = inc + o;
    }
    if (lane == 31) part[warp] = inc;
    const int bad = __syncthreads_or(code);
    if (warp == 0) {
        Sum3 w = part[lane < T / 32 ? lane : 0];
#pragma unroll
        for (int d = 1; d < T / 32; d <<= 1) {
            const Sum3 o = shfl_up(w, d);
            if (lane >= d) w = w + o;
        }
        if (lane < T / 32) part[lane] = w;
    }
    __syncthreads();
    if (warp > 0) inc = inc + part[warp - 1];
    const Sum3 all = part[T / 32 - 1];
    const int count = p.pool[SPEC_POOL_FREE];
    int err = bad;
    if (!err && all.rows > p.row_cap) err = SPEC_PAGED_BAD_ROWS;
    if (!err && (count < 0 || (long long)count + all.rel > p.num_pages || all.alc > (long long)count + all.rel))
        err = SPEC_PAGED_NO_PAGES;
    if (tid < p.nseq) {
        rel[tid + 1] = inc.rel;
        alc[tid + 1] = inc.alc;
        row[tid + 1] = err ? 0 : (int)inc.rows;
        if (blockIdx.x == 0) p.row_start[tid + 1] = err ? 0 : (int)inc.rows;
    }
    if (tid == 0) {
        rel[0] = alc[0] = row[0] = 0;
        if (blockIdx.x == 0) p.row_start[0] = 0;
    }
    __syncthreads();
    if (!err) {
        int* stack = p.pool + SPEC_POOL_HEADER;
        const int R = all.rel, A = all.alc;
        const int t0 = blockIdx.x * T + tid, step = gridDim.x * T;
        constexpr int kGroup = 4;
        const bool aligned = (reinterpret_cast<uintptr_t>(p.slots) & 15) == 0;
        auto entry = [&](int q, int j) -> int& { return p.tables[(size_t)q * p.table_pages + j]; };
        auto released = [&](int i) {
            const int q = owner(rel, p.nseq, i);
            return entry(q, need[q] + i - rel[q]);
        };
        auto taken = [&](int k) {
            const int at = count + R - 1 - k;
            return at < count ? stack[at] : released(at - count);
        };
        // a page as the slots use it: one outside the pool is reported, and its slots lie
        // behind the pool, where the append refuses them (page * 64 could wrap into it)
        auto checked = [&](int page) {
            if ((unsigned)page < (unsigned)p.num_pages) return page;
            atomicCAS(p.pool + SPEC_POOL_ERROR, 0, SPEC_PAGED_BAD_PAGE);
            return p.num_pages;
        };
        for (int i = t0; i < R; i += step) {
            const int page = released(i);
            stack[count + i] = page;
            checked(page);
        }
        for (int k = t0; k < A; k += step) {
            const int q = owner(alc, p.nseq, k);
            entry(q, held[q] + k - alc[q]) = taken(k);
        }
        // slots, kGroup consecutive rows a thread step: their sequence is looked for
        // once and a page once per page
        const int rows = (int)all.rows;
        for (long long g = (long long)t0 * kGroup; g < rows; g += (long long)step * kGroup) {
            const int r0 = (int)g, n = min(kGroup, rows - r0);
            int q = owner(row, p.nseq, r0), at = -1, base = 0;   // at: the page's index in the table row
            int slot[kGroup];
#pragma unroll
            for (int e = 0; e < kGroup; ++e) {
                if (e >= n) break;
                while (row[q + 1] <= r0 + e) {
                    ++q;
                    at = -1;
                }
                const int pos = keep[q] + r0 + e - row[q], j = pos / SPEC_PAGE;
                if (j != at) {
                    at = j;
                    base = checked(j < held[q] ? entry(q, j) : taken(alc[q] + j - held[q])) * SPEC_PAGE;
                }
                slot[e] = base + pos % SPEC_PAGE;
            }
            if (n == kGroup && aligned) {
                *reinterpret_cast<int4*>(p.slots + r0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            } else {
#pragma unroll
                for (int e = 0; e < kGroup; ++e)
                    if (e < n) p.slots[r0 + e] = slot[e];
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        last = 1;
        if (gridDim.x > 1) {
            __threadfence();
            last = atomicInc(reinterpret_cast<unsigned*>(p.pool + kPoolTicket), gridDim.x - 1) == gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!last) return;
    if (!err && tid < p.nseq) p.len[tid] = newlen;
    if (tid == 0) {
        if (!err) p.pool[SPEC_POOL_FREE] = count + all.rel - all.alc;
        else if (p.pool[SPEC_POOL_ERROR] == 0) p.pool[SPEC_POOL_ERROR] = err;
    }
}

__global__ void __launch_bounds__(256) pages_init_kernel(int* pool, int num_pages) {
    pdl_wait();
    pdl_launch_dependents();
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i < SPEC_POOL_HEADER) pool[i] = i == SPEC_POOL_FREE ? num_pages : 0;
    if (i < num_pages) pool[SPEC_POOL_HEADER + i] = num_pages - 1 - i;
}

struct AppendParams {
    const uint16_t *k, *v;
    long long k_stride, v_stride;
    const int* slots;
    const int* count;
    int rows, hkv, hd;
    uint16_t *kpool, *vpool;
    int num_pages;
    int* err;
};

// One 16-byte piece of a key row and the same piece of the value row per
// thread step: consecutive threads take consecutive pieces of a row, so reads
// and (per head) writes are contiguous.
__global__ void __launch_bounds__(256) paged_append_kernel(const __grid_constant__ AppendParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int rows = p.count ? min(p.rows, *p.count) : p.rows;
    const int per_head = p.hd >> 3, per = p.hkv * per_head;   // pieces of a row
    const long long total = (long long)rows * per;
    for (long long i = blockIdx.x * 256 + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
        const int r = (int)(i / per), c = (int)(i - (long long)r * per);
        const int slot = p.slots[r];
        if (slot < 0) continue;
        const int page = slot / SPEC_PAGE;
        if (page >= p.num_pages) {
            if (p.err) atomicCAS(p.err, 0, SPEC_PAGED_BAD_PAGE);
            continue;
        }
        const uint4 kk = *reinterpret_cast<const uint4*>(p.k + r * p.k_stride + c * 8);
        const uint4 vv = *reinterpret_cast<const uint4*>(p.v + r * p.v_stride + c * 8);
        const int h = c / per_head;
        const size_t at = (((size_t)page * p.hkv + h) * SPEC_PAGE + slot % SPEC_PAGE) * p.hd + (c - h * per_head) * 8;
        *reinterpret_cast<uint4*>(p.kpool + at) = kk;
        *reinterpret_cast<uint4*>(p.vpool + at) = vv;
    }
}

cudaError_t launch(const void* fn, unsigned grid, unsigned block, cudaStream_t s, void** args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

spec_status bad(const char* msg) {
    set_last_error(msg);
    return SPEC_ERR_INVALID_ARG;
}

spec_status done(cudaError_t e) {
    if (e == cudaSuccess) return SPEC_OK;
    set_last_error(cudaGetErrorString(e));
    return SPEC_ERR_CUDA;
}

bool misaligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

}  // namespace
}  // namespace sv

extern "C" {

using namespace sv;

spec_status spec_pages_init(int32_t* d_pool, int32_t num_pages, void* cuda_stream) {
    if (!d_pool) return bad("spec_pages_init: null pointer");
    if (misaligned(d_pool, 4)) return bad("spec_pages_init: d_pool is not 4-byte aligned");
    if (num_pages < 1 || num_pages > SPEC_MAX_PAGES) return bad("spec_pages_init: num_pages must be in 1..33554431");
    void* args[] = {&d_pool, &num_pages};
    return done(launch((const void*)pages_init_kernel, (unsigned)((num_pages + 255) / 256), 256,
                       static_cast<cudaStream_t>(cuda_stream), args));
}

spec_status spec_pages_step(int32_t* d_pool, int32_t num_pages, int32_t* d_tables, int32_t table_pages, int32_t* d_len,
                            const int32_t* d_keep, const int32_t* d_add, int32_t nseq, int32_t* d_row_start,
                            int32_t* d_slots, int32_t row_cap, void* cuda_stream) {
    if (nseq < 0 || nseq > SPEC_MAX_SEQS) return bad("spec_pages_step: nseq must be in 0..1024");
    if (num_pages < 1 || num_pages > SPEC_MAX_PAGES) return bad("spec_pages_step: num_pages must be in 1..33554431");
    if (table_pages < 1 || table_pages > SPEC_MAX_TABLE) return bad("spec_pages_step: table_pages must be in 1..1048576");
    if (row_cap < 0) return bad("spec_pages_step: negative row_cap");
    if (nseq == 0) return SPEC_OK;
    if (!d_pool || !d_tables || !d_len || !d_keep || !d_add || !d_row_start || (row_cap > 0 && !d_slots))
        return bad("spec_pages_step: null pointer");
    if (misaligned(d_pool, 4) || misaligned(d_tables, 4) || misaligned(d_len, 4) || misaligned(d_keep, 4) ||
        misaligned(d_add, 4) || misaligned(d_row_start, 4) || misaligned(d_slots, 4))
        return bad("spec_pages_step: a pointer is not 4-byte aligned");
    StepParams p{d_pool, num_pages, d_tables, table_pages, d_len, d_keep, d_add, nseq, d_row_start, d_slots, row_cap};
    // Few sequences and rows: a small CTA starts and synchronises sooner (30 or 128
    // sequences of 4 rows 3.0 us against 3.5 with 1024 threads, one sequence 2.5
    // against 2.9).  Else one CTA up to 4096 rows (4 a thread), then more, up to two
    // per SM: the 2 million slots of 1024 prompts take 9.9 us (16.3 with one row a
    // thread step on 128 CTAs), a verify cycle of 200 sequences 3.7.  Pages that change
    // hands are looked for one by one: 14.2 us with 21600 of them, 7.5 for 200 sequences
    // admitted and retired in turn (12100 pages, 385 thousand slots), 4.2 where 19 of 200
    // blocks pass a page's end.
    void* args[] = {&p};
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    if (nseq <= kFewThreads && row_cap <= 4 * kFewThreads)
        return done(launch((const void*)pages_step_kernel<kFewThreads>, 1, kFewThreads, s, args));
    int grid = row_cap / (4 * kStepThreads) + (row_cap % (4 * kStepThreads) != 0);
    grid = grid < 1 ? 1 : grid > 304 ? 304 : grid;
    return done(launch((const void*)pages_step_kernel<kStepThreads>, (unsigned)grid, kStepThreads, s, args));
}

spec_status spec_paged_append(const void* d_k, int64_t k_stride, const void* d_v, int64_t v_stride, const int32_t* d_slots,
                              const int32_t* d_row_count_opt, int32_t rows, int32_t n_kv_heads, int32_t head_dim,
                              void* d_kpool, void* d_vpool, int32_t num_pages, int32_t* d_error_opt, void* cuda_stream) {
    if (rows < 0) return bad("spec_paged_append: negative rows");
    if (head_dim != 64 && head_dim != 128) return bad("spec_paged_append: head_dim must be 64 or 128");
    if (n_kv_heads < 1 || n_kv_heads > 1024) return bad("spec_paged_append: n_kv_heads must be in 1..1024");
    if (num_pages < 1 || num_pages > SPEC_MAX_PAGES) return bad("spec_paged_append: num_pages must be in 1..33554431");
    const int64_t row = (int64_t)n_kv_heads * head_dim;
    if (k_stride < row || v_stride < row || (k_stride & 7) || (v_stride & 7))
        return bad("spec_paged_append: row strides must be multiples of 8 and at least n_kv_heads * head_dim");
    if (rows == 0) return SPEC_OK;
    if (!d_k || !d_v || !d_slots || !d_kpool || !d_vpool) return bad("spec_paged_append: null pointer");
    if (misaligned(d_k, 16) || misaligned(d_v, 16) || misaligned(d_kpool, 16) || misaligned(d_vpool, 16))
        return bad("spec_paged_append: keys, values and pools must be 16-byte aligned");
    if (misaligned(d_slots, 4) || misaligned(d_row_count_opt, 4) || misaligned(d_error_opt, 4))
        return bad("spec_paged_append: an int32 pointer is not 4-byte aligned");
    AppendParams p{static_cast<const uint16_t*>(d_k), static_cast<const uint16_t*>(d_v), k_stride, v_stride, d_slots,
                   d_row_count_opt, rows, n_kv_heads, head_dim, static_cast<uint16_t*>(d_kpool),
                   static_cast<uint16_t*>(d_vpool), num_pages, d_error_opt};
    const int64_t pieces = (int64_t)rows * n_kv_heads * (head_dim / 8);
    const int64_t want = (pieces + 255) / 256;
    const int sms = current_sms();
    if (!sms) {
        set_last_error("spec_paged_append: no current CUDA device");
        return SPEC_ERR_CUDA;
    }
    const unsigned grid = (unsigned)(want < 8 * sms ? want : 8 * sms);
    void* args[] = {&p};
    return done(launch((const void*)paged_append_kernel, grid, 256, static_cast<cudaStream_t>(cuda_stream), args));
}

}  // extern "C"
