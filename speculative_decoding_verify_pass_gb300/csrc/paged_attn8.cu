// Attention of each sequence's newest positions over the 8-bit paged cache:
// a warp for each (row, query head), the softmax's maximum and sum running.
#include <math.h>

#include "internal.h"
#include "paged_split.h"
#include "spec.h"

namespace sv {
namespace {

struct Paged8Params {
    const uint16_t* q;
    long long q_stride;
    const int *row_start, *len, *tables;
    int table_pages, nseq, rows, hq, hkv;
    float scale_log2;
    const uint8_t *kpool, *vpool, *scales;
    int num_pages;
    uint16_t* out;
    long long out_stride;
    int* err;
};

__device__ __forceinline__ float pow2_byte(int b) {
    return b == 0 ? __uint_as_float(1u << 22) : b == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)b << 23);
}
// Two e4m3 codes (the low two bytes) as floats.
__device__ __forceinline__ float2 e4m3x2(uint32_t x) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)x));
    float2 f;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(f.x), "=f"(f.y) : "r"(h));
    return f;
}

template <int HD>
__global__ void __launch_bounds__(256) paged8_kernel(const __grid_constant__ Paged8Params p) {
    constexpr int V = HD / 32;
    const int lane = threadIdx.x & 31;
    const int i = (blockIdx.x * 256 + threadIdx.x) >> 5;
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x == 0 && p.err)
        for (int q = threadIdx.x; q < p.nseq; q += 256) {
            const int r0 = p.row_start[q], r1 = p.row_start[q + 1], n = p.len[q];
            const bool bad_rows = r0 < 0 || r1 < r0 || r1 > p.rows;
            if (bad_rows || n < 0 || n > (long long)p.table_pages * SPEC_PAGE)
                atomicCAS(p.err, 0, bad_rows ? SPEC_PAGED_BAD_ROWS : SPEC_PAGED_BAD_LENGTH);
        }
    const int row = i / p.hq, h = i - row * p.hq;
    if (row >= p.rows) return;
    int b = 0;
    while (b < p.nseq && !(p.row_start[b] <= row && row < p.row_start[b + 1])) ++b;
    if (b == p.nseq) return;
    const int r0 = p.row_start[b], r1 = p.row_start[b + 1], n = p.len[b];
    if (r0 < 0 || r1 > p.rows || n < 0 || n > (long long)p.table_pages * SPEC_PAGE) return;
    const int last = n - (r1 - row);
    const int kvh = h / (p.hq / p.hkv);
    float q[V], o[V] = {}, m = -INFINITY, l = 0.f;
    for (int e = 0; e < V; ++e) q[e] = bf2f(p.q[row * p.q_stride + (long long)h * HD + lane * V + e]);
    for (int t = 0; t <= last; ++t) {
        const int page = p.tables[(size_t)b * p.table_pages + t / SPEC_PAGE];
        const bool ok = page >= 0 && page < p.num_pages;
        if (!ok && p.err) atomicCAS(p.err, 0, SPEC_PAGED_BAD_PAGE);
        const size_t ph = ok ? (size_t)page * p.hkv + kvh : 0, at = (ph * SPEC_PAGE + t % SPEC_PAGE) * HD + lane * V;
        uint32_t kc, vc;
        if constexpr (V == 4) kc = *reinterpret_cast<const uint32_t*>(p.kpool + at), vc = *reinterpret_cast<const uint32_t*>(p.vpool + at);
        else kc = *reinterpret_cast<const uint16_t*>(p.kpool + at), vc = *reinterpret_cast<const uint16_t*>(p.vpool + at);
        const float ks = pow2_byte(p.scales[ph * 2 * SPEC_PAGE + t % SPEC_PAGE]), vs = pow2_byte(p.scales[ph * 2 * SPEC_PAGE + SPEC_PAGE + t % SPEC_PAGE]);
        if (!ok) kc = vc = 0;
        float s = 0.f, v[V];
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float2 k2 = e4m3x2(kc >> (8 * e)), v2 = e4m3x2(vc >> (8 * e));
            s += q[e] * k2.x + q[e + 1] * k2.y;
            v[e] = v2.x * vs, v[e + 1] = v2.y * vs;
        }
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= (ok ? ks : 1.f) * p.scale_log2;
        const float now = fmaxf(m, s), f = m == now ? 1.f : exp2f(m - now), w = s == -INFINITY ? 0.f : exp2f(s - now);
        m = now;
        l = l * f + w;
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = o[e] * f + w * (ok ? v[e] : 0.f);
    }
    for (int e = 0; e < V; ++e)
        p.out[row * p.out_stride + (long long)h * HD + lane * V + e] = f2bf(last >= 0 ? o[e] / l : 0.f);
}

spec_status bad(const char* msg) {
    set_last_error(msg);
    return SPEC_ERR_INVALID_ARG;
}

bool misaligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

const char* head_error(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t max_new) {
    if (head_dim != 64 && head_dim != 128) return "spec_paged_attention_fp8: head_dim must be 64 or 128";
    if (n_kv_heads < 1 || n_kv_heads > 1024 || n_heads < n_kv_heads || n_heads % n_kv_heads)
        return "spec_paged_attention_fp8: n_heads must be a multiple of n_kv_heads, 1..1024";
    if (n_heads / n_kv_heads > 128) return "spec_paged_attention_fp8: at most 128 query heads per kv head";
    if (max_new < 1) return "spec_paged_attention_fp8: max_new must be at least 1";
    return nullptr;
}

}  // namespace
}  // namespace sv

extern "C" {

using namespace sv;

spec_status spec_paged_attention_fp8_workspace(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t max_new,
                                               int32_t table_pages, size_t* out_bytes) {
    if (!out_bytes) return bad("spec_paged_attention_fp8_workspace: null pointer");
    if (const char* e = head_error(n_heads, n_kv_heads, head_dim, max_new)) return bad(e);
    if (table_pages < 1 || table_pages > SPEC_MAX_TABLE) return bad("spec_paged_attention_fp8: table_pages must be in 1..1048576");
    *out_bytes = 0;
    return SPEC_OK;
}

spec_status spec_paged_attention_fp8(const void* d_q, int64_t q_stride, const int32_t* d_row_start, const int32_t* d_len,
                                     const int32_t* d_tables, int32_t table_pages, int32_t nseq, int32_t rows,
                                     int32_t max_new, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, float scale,
                                     const void* d_kpool, const void* d_vpool, const void* d_scales, int32_t num_pages,
                                     void* d_out, int64_t out_stride, int32_t* d_error_opt, void* d_work, size_t work_bytes,
                                     void* cuda_stream) {
    if (const char* e = head_error(n_heads, n_kv_heads, head_dim, max_new)) return bad(e);
    if (nseq < 0 || nseq > SPEC_MAX_SEQS) return bad("spec_paged_attention_fp8: nseq must be in 0..1024");
    if (rows < 0) return bad("spec_paged_attention_fp8: negative rows");
    if (table_pages < 1 || table_pages > SPEC_MAX_TABLE) return bad("spec_paged_attention_fp8: table_pages must be in 1..1048576");
    if (num_pages < 1 || num_pages > SPEC_MAX_PAGES) return bad("spec_paged_attention_fp8: num_pages must be in 1..33554431");
    if ((int64_t)num_pages * n_kv_heads > 0x7fffffff) return bad("spec_paged_attention_fp8: num_pages * n_kv_heads must fit int32");
    if (!(scale > 0.f) || !isfinite(scale)) return bad("spec_paged_attention_fp8: scale must be positive and finite");
    const int64_t row = (int64_t)n_heads * head_dim;
    if (q_stride < row || out_stride < row || (q_stride & 7) || (out_stride & 7) || q_stride >= (1ll << 38) ||
        out_stride >= (1ll << 38))
        return bad("spec_paged_attention_fp8: row strides must be multiples of 8, at least n_heads * head_dim and below 2^38");
    if (nseq == 0 || rows == 0) return SPEC_OK;
    if (!d_q || !d_row_start || !d_len || !d_tables || !d_kpool || !d_vpool || !d_scales || !d_out)
        return bad("spec_paged_attention_fp8: null pointer");
    if (misaligned(d_q, 16) || misaligned(d_out, 16) || misaligned(d_kpool, 16) || misaligned(d_vpool, 16) || misaligned(d_scales, 16))
        return bad("spec_paged_attention_fp8: queries, output, pools and scales must be 16-byte aligned");
    if (misaligned(d_row_start, 4) || misaligned(d_len, 4) || misaligned(d_tables, 4) || misaligned(d_error_opt, 4))
        return bad("spec_paged_attention_fp8: an int32 pointer is not 4-byte aligned");
    Paged8Params p{static_cast<const uint16_t*>(d_q), q_stride, d_row_start, d_len, d_tables, table_pages, nseq, rows, n_heads,
                   n_kv_heads, scale * 1.44269504088896340736f, static_cast<const uint8_t*>(d_kpool),
                   static_cast<const uint8_t*>(d_vpool), static_cast<const uint8_t*>(d_scales), num_pages,
                   static_cast<uint16_t*>(d_out), out_stride, d_error_opt};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((int64_t)rows * n_heads + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = static_cast<cudaStream_t>(cuda_stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {&p};
    const cudaError_t e = cudaLaunchKernelExC(&cfg, head_dim == 128 ? (const void*)paged8_kernel<128> : (const void*)paged8_kernel<64>, args);
    if (e == cudaSuccess) return SPEC_OK;
    set_last_error(cudaGetErrorString(e));
    return SPEC_ERR_CUDA;
}

}  // extern "C"
