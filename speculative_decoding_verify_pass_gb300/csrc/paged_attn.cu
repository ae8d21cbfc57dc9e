// Attention of each sequence's newest positions over a paged cache.
//
// One warp per (row, query head): an online softmax over the row's visible
// positions, keys and values read from their pages.
#include <math.h>
#include <stdio.h>

#include "internal.h"
#include "spec.h"

namespace sv {
namespace {

struct PagedParams {
    const uint16_t* q;
    long long q_stride;
    const int *row_start, *len, *tables;
    int table_pages, nseq, rows, hq, hkv;
    float scale;
    const uint16_t *kpool, *vpool;
    int num_pages;
    uint16_t* out;
    long long out_stride;
    int* err;
};

template <int HD>
__global__ void __launch_bounds__(128) paged_attn_simple_kernel(const __grid_constant__ PagedParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int q = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r0 = p.row_start[q], r1 = p.row_start[q + 1], len = p.len[q];
    const bool bad_rows = r0 < 0 || r1 < r0 || r1 > p.rows, bad_len = len < 0 || len > (long long)p.table_pages * SPEC_PAGE;
    if (bad_rows || bad_len) {
        if (p.err) atomicCAS(p.err, 0, bad_rows ? SPEC_PAGED_BAD_ROWS : SPEC_PAGED_BAD_LENGTH);
        return;
    }
    constexpr int V = HD / 32;
    const int kvh = h / (p.hq / p.hkv);
    for (int r = r0 + warp; r < r1; r += 4) {
        const int seen = len - (r1 - r0) + (r - r0) + 1;
        float qv[V], o[V], m = -INFINITY, l = 0.f;
        for (int e = 0; e < V; ++e) {
            qv[e] = bf2f(p.q[r * p.q_stride + (long long)h * HD + lane * V + e]) * p.scale;
            o[e] = 0.f;
        }
        for (int i = 0; i < seen; ++i) {
            const int page = p.tables[(size_t)q * p.table_pages + i / SPEC_PAGE];
            float kk[V], vv[V], s = 0.f;
            const bool ok = page >= 0 && page < p.num_pages;
            if (!ok && p.err && lane == 0) atomicCAS(p.err, 0, SPEC_PAGED_BAD_PAGE);
            const size_t at = ok ? (((size_t)page * p.hkv + kvh) * SPEC_PAGE + i % SPEC_PAGE) * HD + lane * V : 0;
            for (int e = 0; e < V; ++e) {
                kk[e] = ok ? bf2f(p.kpool[at + e]) : 0.f;
                vv[e] = ok ? bf2f(p.vpool[at + e]) : 0.f;
                s += qv[e] * kk[e];
            }
            for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            const float mn = fmaxf(m, s), w = m == mn ? 1.f : expf(m - mn), a = expf(s - mn);
            l = l * w + a;
            for (int e = 0; e < V; ++e) o[e] = o[e] * w + a * vv[e];
            m = mn;
        }
        for (int e = 0; e < V; ++e)
            p.out[r * p.out_stride + (long long)h * HD + lane * V + e] = f2bf(seen > 0 ? o[e] / l : 0.f);
    }
}

spec_status bad(const char* msg) {
    set_last_error(msg);
    return SPEC_ERR_INVALID_ARG;
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

}  // namespace
}  // namespace sv

extern "C" {

using namespace sv;

spec_status spec_paged_attention_workspace(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t max_new,
                                           size_t* out_bytes) {
    if (!out_bytes) return bad("spec_paged_attention_workspace: null pointer");
    if (const char* e = head_error(n_heads, n_kv_heads, head_dim, max_new)) return bad(e);
    *out_bytes = 256;
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
    if (q_stride < row || out_stride < row || (q_stride & 7) || (out_stride & 7))
        return bad("spec_paged_attention: row strides must be multiples of 8 and at least n_heads * head_dim");
    if (nseq == 0 || rows == 0) return SPEC_OK;
    if (!d_q || !d_row_start || !d_len || !d_tables || !d_kpool || !d_vpool || !d_out || !d_work)
        return bad("spec_paged_attention: null pointer");
    if (misaligned(d_q, 16) || misaligned(d_out, 16) || misaligned(d_kpool, 16) || misaligned(d_vpool, 16))
        return bad("spec_paged_attention: queries, output and pools must be 16-byte aligned");
    if (misaligned(d_row_start, 4) || misaligned(d_len, 4) || misaligned(d_tables, 4) || misaligned(d_error_opt, 4))
        return bad("spec_paged_attention: an int32 pointer is not 4-byte aligned");
    if (misaligned(d_work, 256)) return bad("spec_paged_attention: d_work is not 256-byte aligned");
    if (work_bytes < 256) return bad("spec_paged_attention: work_bytes is less than the workspace these heads need");
    PagedParams p{static_cast<const uint16_t*>(d_q), q_stride, d_row_start, d_len, d_tables, table_pages, nseq, rows,
                  n_heads, n_kv_heads, scale, static_cast<const uint16_t*>(d_kpool), static_cast<const uint16_t*>(d_vpool),
                  num_pages, static_cast<uint16_t*>(d_out), out_stride, d_error_opt};
    const dim3 grid((unsigned)nseq, (unsigned)n_heads);
    if (head_dim == 128) paged_attn_simple_kernel<128><<<grid, 128, 0, static_cast<cudaStream_t>(cuda_stream)>>>(p);
    else paged_attn_simple_kernel<64><<<grid, 128, 0, static_cast<cudaStream_t>(cuda_stream)>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return SPEC_OK;
    set_last_error(cudaGetErrorString(e));
    return SPEC_ERR_CUDA;
}

}  // extern "C"
