// The 8-bit paged cache's append and read.
//
// A row of a kv head, x[hd], is kept as e4m3 codes c and one exponent e:
//     e = the least integer with max |x| <= 448 * 2^e, at least -126 (max over finite x)
//     c = x * 2^-e rounded to the nearest e4m3, ties to even
// kept as the byte e + 127.  The scale is a power of two, so that x * 2^-e and
// c * 2^e are exact: the only rounding is the one to 4 significant bits (2^-4 of
// the value, 2^-10 of 2^e below 2^-6 of it), and what is read back is the value that
// attention sees.  It belongs to one position, so that writing a position says
// nothing about others: a rejected draft leaves no trace in the tokens before it.
// Infinities and NaN become NaN.
//
// Both are bound by memory (4 bytes in and 2 out per pair of elements, or the
// other way): a thread takes 8 elements of the key row and the same 8 of the value
// row, the 8 or 16 threads of a head find the two maxima with shuffles.
#include <cuda_fp8.h>
#include <stdio.h>

#include "internal.h"
#include "spec.h"

namespace sv {
namespace {

struct Pools8 {
    uint8_t *k, *v, *scales;    // [page][hkv][64][hd] twice, [page][hkv][2][64]
    int num_pages, hkv, hd;
};

struct Rows8Params {
    uint16_t *k, *v;            // bf16 rows: read by the append, written by the read
    long long k_stride, v_stride;
    const int *slots, *count;
    int rows;
    Pools8 pool;
    int* err;
};

// Exponent byte of a row whose largest finite magnitude has the bf16 bits `top`.
// 448 = 1.75 * 2^8: a significand above 1.75 takes one more.
__device__ __forceinline__ int scale_byte(uint32_t top) {
    const int e = (int)(top >> 7) - 8 + ((top & 0x7F) > 0x60);      // + 127
    return max(e, 1);
}
__device__ __forceinline__ float scale_of(int byte) {               // 2^(byte - 127); 255: NaN
    return byte == 0 ? __uint_as_float(1u << 22) : byte == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)byte << 23);
}

// The larger of two bf16 magnitudes among finite ones, for both halves of x.
__device__ __forceinline__ uint32_t top_of(uint32_t top, uint32_t x) {
    const uint32_t lo = x & 0x7FFFu, hi = (x >> 16) & 0x7FFFu;
    if (lo < 0x7F80u) top = max(top, lo);
    if (hi < 0x7F80u) top = max(top, hi);
    return top;
}

// Two bf16 times inv as e4m3 codes (infinities as NaN), the low one in the low byte.
__device__ __forceinline__ uint32_t codes(uint32_t x, float inv) {
    const float a = __uint_as_float(x << 16), b = __uint_as_float(x & 0xFFFF0000u);
    const float nan = __uint_as_float(0x7FC00000u);
    const float2 f = make_float2(isinf(a) ? nan : a * inv, isinf(b) ? nan : b * inv);
    return __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
}

// The row's place in the pools, (page * hkv + head), or -1: skipped, or outside the
// pool (reported).
__device__ __forceinline__ long long page_head(const Rows8Params& p, int slot, int h) {
    if (slot < 0) return -1;
    const int page = slot / SPEC_PAGE;
    if (page >= p.pool.num_pages) {
        if (p.err) atomicCAS(p.err, 0, SPEC_PAGED_BAD_PAGE);
        return -1;
    }
    return (long long)page * p.pool.hkv + h;
}

__global__ void __launch_bounds__(256) append8_kernel(const __grid_constant__ Rows8Params p) {
    pdl_wait();
    pdl_launch_dependents();
    const int rows = p.count ? min(p.rows, *p.count) : p.rows;
    const int per_head = p.pool.hd >> 3, per = p.pool.hkv * per_head;    // threads of a head: 8 or 16
    const long long total = (long long)rows * per, step = (long long)gridDim.x * 256;
    // whole warps go round together: the shuffles below name every lane
    for (long long i0 = blockIdx.x * 256; i0 < total; i0 += step) {
        const long long i = i0 + threadIdx.x;
        const int r = (int)(min(i, total - 1) / per), c = (int)(min(i, total - 1) - (long long)r * per), h = c / per_head, d = c - h * per_head;
        const int slot = i < total ? p.slots[r] : -1;
        const long long at = page_head(p, slot, h);
        uint4 kk = {}, vv = {};
        if (at >= 0) {
            kk = *reinterpret_cast<const uint4*>(p.k + r * p.k_stride + c * 8);
            vv = *reinterpret_cast<const uint4*>(p.v + r * p.v_stride + c * 8);
        }
        uint32_t kt = top_of(top_of(top_of(top_of(0, kk.x), kk.y), kk.z), kk.w);
        uint32_t vt = top_of(top_of(top_of(top_of(0, vv.x), vv.y), vv.z), vv.w);
        uint32_t both = kt << 16 | vt;          // bf16 magnitudes: 15 bits each
        for (int m = 1; m < per_head; m <<= 1) {
            const uint32_t o = __shfl_xor_sync(0xffffffffu, both, m);
            both = max(both & 0xFFFF0000u, o & 0xFFFF0000u) | max(both & 0xFFFFu, o & 0xFFFFu);
        }
        if (at < 0) continue;
        const int kb = scale_byte(both >> 16), vb = scale_byte(both & 0xFFFFu), t = slot % SPEC_PAGE;
        const float ki = __uint_as_float((uint32_t)(254 - kb) << 23), vi = __uint_as_float((uint32_t)(254 - vb) << 23);
        const size_t to = ((size_t)at * SPEC_PAGE + t) * p.pool.hd + d * 8;
        *reinterpret_cast<uint2*>(p.pool.k + to) = make_uint2(codes(kk.x, ki) | codes(kk.y, ki) << 16, codes(kk.z, ki) | codes(kk.w, ki) << 16);
        *reinterpret_cast<uint2*>(p.pool.v + to) = make_uint2(codes(vv.x, vi) | codes(vv.y, vi) << 16, codes(vv.z, vi) | codes(vv.w, vi) << 16);
        if (d == 0) {
            uint8_t* s = p.pool.scales + (size_t)at * 2 * SPEC_PAGE + t;
            s[0] = (uint8_t)kb;
            s[SPEC_PAGE] = (uint8_t)vb;
        }
    }
}

// Two codes (the low two bytes) times scale, as bf16.
__device__ __forceinline__ uint32_t values(uint32_t x, float scale) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)x, __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * scale, f.y * scale);
    return *reinterpret_cast<const uint32_t*>(&b);
}

__global__ void __launch_bounds__(256) read8_kernel(const __grid_constant__ Rows8Params p) {
    pdl_wait();
    pdl_launch_dependents();
    const int rows = p.count ? min(p.rows, *p.count) : p.rows;
    const int per_head = p.pool.hd >> 3, per = p.pool.hkv * per_head;
    const long long total = (long long)rows * per;
    for (long long i = blockIdx.x * 256 + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
        const int r = (int)(i / per), c = (int)(i - (long long)r * per), h = c / per_head, d = c - h * per_head;
        const int slot = p.slots[r];
        const long long at = page_head(p, slot, h);
        if (at < 0) continue;
        const int t = slot % SPEC_PAGE;
        const size_t from = ((size_t)at * SPEC_PAGE + t) * p.pool.hd + d * 8;
        const uint2 kk = *reinterpret_cast<const uint2*>(p.pool.k + from), vv = *reinterpret_cast<const uint2*>(p.pool.v + from);
        const uint8_t* s = p.pool.scales + (size_t)at * 2 * SPEC_PAGE + t;
        const float ks = scale_of(s[0]), vs = scale_of(s[SPEC_PAGE]);
        *reinterpret_cast<uint4*>(p.k + r * p.k_stride + c * 8) =
            make_uint4(values(kk.x & 0xFFFFu, ks), values(kk.x >> 16, ks), values(kk.y & 0xFFFFu, ks), values(kk.y >> 16, ks));
        *reinterpret_cast<uint4*>(p.v + r * p.v_stride + c * 8) =
            make_uint4(values(vv.x & 0xFFFFu, vs), values(vv.x >> 16, vs), values(vv.y & 0xFFFFu, vs), values(vv.y >> 16, vs));
    }
}

spec_status bad(const char* call, const char* what) {
    static thread_local char msg[160];
    snprintf(msg, sizeof msg, "%s: %s", call, what);
    set_last_error(msg);
    return SPEC_ERR_INVALID_ARG;
}

bool misaligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// Checks and launches either call.
spec_status run(const char* call, const void* fn, const void* d_k, int64_t k_stride, const void* d_v, int64_t v_stride,
                const int32_t* d_slots, const int32_t* d_row_count_opt, int32_t rows, int32_t n_kv_heads, int32_t head_dim,
                const void* d_kpool, const void* d_vpool, const void* d_scales, int32_t num_pages, int32_t* d_error_opt,
                void* cuda_stream) {
    if (rows < 0) return bad(call, "negative rows");
    if (head_dim != 64 && head_dim != 128) return bad(call, "head_dim must be 64 or 128");
    if (n_kv_heads < 1 || n_kv_heads > 1024) return bad(call, "n_kv_heads must be in 1..1024");
    if (num_pages < 1 || num_pages > SPEC_MAX_PAGES) return bad(call, "num_pages must be in 1..33554431");
    const int64_t row = (int64_t)n_kv_heads * head_dim;
    if (k_stride < row || v_stride < row || (k_stride & 7) || (v_stride & 7) || k_stride >= (1ll << 38) || v_stride >= (1ll << 38))
        return bad(call, "row strides must be multiples of 8, at least n_kv_heads * head_dim and below 2^38");
    if (rows == 0) return SPEC_OK;
    if (!d_k || !d_v || !d_slots || !d_kpool || !d_vpool || !d_scales) return bad(call, "null pointer");
    if (misaligned(d_k, 16) || misaligned(d_v, 16) || misaligned(d_kpool, 16) || misaligned(d_vpool, 16) || misaligned(d_scales, 16))
        return bad(call, "keys, values, pools and scales must be 16-byte aligned");
    if (misaligned(d_slots, 4) || misaligned(d_row_count_opt, 4) || misaligned(d_error_opt, 4))
        return bad(call, "an int32 pointer is not 4-byte aligned");
    Rows8Params p;
    p.k = static_cast<uint16_t*>(const_cast<void*>(d_k));
    p.v = static_cast<uint16_t*>(const_cast<void*>(d_v));
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.slots = d_slots;
    p.count = d_row_count_opt;
    p.rows = rows;
    p.pool.k = static_cast<uint8_t*>(const_cast<void*>(d_kpool));
    p.pool.v = static_cast<uint8_t*>(const_cast<void*>(d_vpool));
    p.pool.scales = static_cast<uint8_t*>(const_cast<void*>(d_scales));
    p.pool.num_pages = num_pages;
    p.pool.hkv = n_kv_heads;
    p.pool.hd = head_dim;
    p.err = d_error_opt;
    const int64_t want = ((int64_t)rows * n_kv_heads * (head_dim / 8) + 255) / 256;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(want < 8 * 152 ? want : 8 * 152));
    cfg.blockDim = dim3(256);
    cfg.stream = static_cast<cudaStream_t>(cuda_stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {&p};
    const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
    if (e == cudaSuccess) return SPEC_OK;
    set_last_error(cudaGetErrorString(e));
    return SPEC_ERR_CUDA;
}

}  // namespace
}  // namespace sv

extern "C" {

using namespace sv;

spec_status spec_paged_append_fp8(const void* d_k, int64_t k_stride, const void* d_v, int64_t v_stride, const int32_t* d_slots,
                                  const int32_t* d_row_count_opt, int32_t rows, int32_t n_kv_heads, int32_t head_dim,
                                  void* d_kpool, void* d_vpool, void* d_scales, int32_t num_pages, int32_t* d_error_opt,
                                  void* cuda_stream) {
    return run("spec_paged_append_fp8", (const void*)append8_kernel, d_k, k_stride, d_v, v_stride, d_slots, d_row_count_opt, rows,
               n_kv_heads, head_dim, d_kpool, d_vpool, d_scales, num_pages, d_error_opt, cuda_stream);
}

spec_status spec_paged_read_fp8(const int32_t* d_slots, const int32_t* d_row_count_opt, int32_t rows, int32_t n_kv_heads,
                                int32_t head_dim, const void* d_kpool, const void* d_vpool, const void* d_scales,
                                int32_t num_pages, void* d_k, int64_t k_stride, void* d_v, int64_t v_stride,
                                int32_t* d_error_opt, void* cuda_stream) {
    return run("spec_paged_read_fp8", (const void*)read8_kernel, d_k, k_stride, d_v, v_stride, d_slots, d_row_count_opt, rows,
               n_kv_heads, head_dim, d_kpool, d_vpool, d_scales, num_pages, d_error_opt, cuda_stream);
}

}  // extern "C"
