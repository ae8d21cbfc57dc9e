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
// row, the 8 or 16 threads of a head find the two maxima with shuffles.  So that
// issue does not bound them first, a thread walks its items without divisions, and
// maxima and infinities are looked for in pairs of halves (28.7 us -> 17.1 for 16001
// rows of 8 x 128 appended; 98 MB: 5.7 TB/s).  Read back, 30011 such rows take 30.6 us
// (6.0 TB/s).  16 elements a thread were slower: 18.0 and 39.7 us.
#include <cuda_fp8.h>
#include <stdio.h>

#include "internal.h"
#include "spec.h"

namespace sv {
namespace {

constexpr int kThreads = 256, kElems = 8;       // of a CTA; of a key row, and of a value row, that a thread takes
constexpr int kCtas = 8;                        // of an SM, at most

struct Pools8 {
    uint8_t *k, *v, *scales;    // [page][hkv][64][hd] twice, [page][hkv][2][64]
    int num_pages, hkv;
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

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The largest finite magnitude (bf16 bits) of 4 words of two bf16 each, in which
// infinities become NaN.
__device__ __forceinline__ uint32_t top_of(uint32_t (&x)[4]) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) m = max_u16x2(m, x[k] & 0x7FFF7FFFu);
    if (((m + 0x00800080u) & 0x80008000u) == 0) return max(m & 0xFFFFu, m >> 16);
    m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t lo = x[k] & 0x7FFFu, hi = (x[k] >> 16) & 0x7FFFu;
        if (lo < 0x7F80u) m = max(m, lo);
        if (hi < 0x7F80u) m = max(m, hi);
        if (lo == 0x7F80u) x[k] |= 0x7Fu;
        if (hi == 0x7F80u) x[k] |= 0x7F0000u;
    }
    return m;
}

// Two bf16 times inv as e4m3 codes, the low one in the low byte.
__device__ __forceinline__ uint32_t codes(uint32_t x, float inv) {
    return __nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(x << 16) * inv, __uint_as_float(x & 0xFFFF0000u) * inv), __NV_SATFINITE, __NV_E4M3);
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

// A thread's items: `per` a row, over all rows in steps of the grid.
struct Items {
    unsigned r, rows;
    int c, step_r, step_c, per;
    __device__ __forceinline__ Items(const Rows8Params& p, int per_) : per(per_) {
        const int n = p.count ? min(p.rows, *p.count) : p.rows;
        rows = n > 0 ? n : 0;
        const int i = blockIdx.x * kThreads + threadIdx.x, step = gridDim.x * kThreads;     // below 2^31: the grid is bounded
        r = i / per;
        c = i - r * per;
        step_r = step / per;
        step_c = step - step_r * per;
    }
    __device__ __forceinline__ bool more() const { return r < rows; }
    __device__ __forceinline__ void step() {
        r += step_r;
        c += step_c;
        if (c >= per) c -= per, ++r;
    }
};

template <int HD>
__global__ void __launch_bounds__(kThreads) append8_kernel(const __grid_constant__ Rows8Params p) {
    constexpr int kPerHead = HD / kElems;       // threads of a head
    pdl_wait();
    pdl_launch_dependents();
    // the threads of a head go round together
    const unsigned lanes = ((1u << kPerHead) - 1u) << (threadIdx.x & 31 & -kPerHead);
#pragma unroll 1
    for (Items it(p, p.pool.hkv * kPerHead); it.more(); it.step()) {
        const int slot = p.slots[it.r], h = it.c / kPerHead, d = it.c % kPerHead;
        // a padding row's are read too: the loads do not wait for its slot
        const uint4 a = *reinterpret_cast<const uint4*>(p.k + it.r * p.k_stride + it.c * kElems);
        const uint4 b = *reinterpret_cast<const uint4*>(p.v + it.r * p.v_stride + it.c * kElems);
        uint32_t k[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
        const long long at = page_head(p, slot, h);
        uint32_t both = top_of(k) << 16;        // bf16 magnitudes: 15 bits each
        both |= top_of(v);
#pragma unroll
        for (int m = 1; m < kPerHead; m <<= 1) both = max_u16x2(both, __shfl_xor_sync(lanes, both, m));
        if (at < 0) continue;
        const int kb = scale_byte(both >> 16), vb = scale_byte(both & 0xFFFFu), t = slot % SPEC_PAGE;
        const float ki = __uint_as_float((uint32_t)(254 - kb) << 23), vi = __uint_as_float((uint32_t)(254 - vb) << 23);
        const size_t to = ((size_t)at * SPEC_PAGE + t) * HD + d * kElems;
        *reinterpret_cast<uint2*>(p.pool.k + to) = make_uint2(codes(k[0], ki) | codes(k[1], ki) << 16, codes(k[2], ki) | codes(k[3], ki) << 16);
        *reinterpret_cast<uint2*>(p.pool.v + to) = make_uint2(codes(v[0], vi) | codes(v[1], vi) << 16, codes(v[2], vi) | codes(v[3], vi) << 16);
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

template <int HD>
__global__ void __launch_bounds__(kThreads) read8_kernel(const __grid_constant__ Rows8Params p) {
    constexpr int kPerHead = HD / kElems;
    pdl_wait();
    pdl_launch_dependents();
#pragma unroll 1
    for (Items it(p, p.pool.hkv * kPerHead); it.more(); it.step()) {
        const int slot = p.slots[it.r], h = it.c / kPerHead, d = it.c % kPerHead;
        const long long at = page_head(p, slot, h);
        if (at < 0) continue;
        const int t = slot % SPEC_PAGE;
        const size_t from = ((size_t)at * SPEC_PAGE + t) * HD + d * kElems;
        const uint2 k = *reinterpret_cast<const uint2*>(p.pool.k + from), v = *reinterpret_cast<const uint2*>(p.pool.v + from);
        const uint8_t* s = p.pool.scales + (size_t)at * 2 * SPEC_PAGE + t;
        const float ks = scale_of(s[0]), vs = scale_of(s[SPEC_PAGE]);
        *reinterpret_cast<uint4*>(p.k + it.r * p.k_stride + it.c * kElems) =
            make_uint4(values(k.x & 0xFFFFu, ks), values(k.x >> 16, ks), values(k.y & 0xFFFFu, ks), values(k.y >> 16, ks));
        *reinterpret_cast<uint4*>(p.v + it.r * p.v_stride + it.c * kElems) =
            make_uint4(values(v.x & 0xFFFFu, vs), values(v.x >> 16, vs), values(v.y & 0xFFFFu, vs), values(v.y >> 16, vs));
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
    p.err = d_error_opt;
    const int sms = current_sms();
    if (!sms) {
        bad(call, "no current CUDA device");
        return SPEC_ERR_CUDA;
    }
    const int64_t most = (int64_t)kCtas * sms, want = ((int64_t)rows * n_kv_heads * (head_dim / kElems) + kThreads - 1) / kThreads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(want < most ? want : most));
    cfg.blockDim = dim3(kThreads);
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
    return run("spec_paged_append_fp8", head_dim == 64 ? (const void*)append8_kernel<64> : (const void*)append8_kernel<128>, d_k, k_stride, d_v, v_stride, d_slots, d_row_count_opt, rows,
               n_kv_heads, head_dim, d_kpool, d_vpool, d_scales, num_pages, d_error_opt, cuda_stream);
}

spec_status spec_paged_read_fp8(const int32_t* d_slots, const int32_t* d_row_count_opt, int32_t rows, int32_t n_kv_heads,
                                int32_t head_dim, const void* d_kpool, const void* d_vpool, const void* d_scales,
                                int32_t num_pages, void* d_k, int64_t k_stride, void* d_v, int64_t v_stride,
                                int32_t* d_error_opt, void* cuda_stream) {
    return run("spec_paged_read_fp8", head_dim == 64 ? (const void*)read8_kernel<64> : (const void*)read8_kernel<128>, d_k, k_stride, d_v, v_stride, d_slots, d_row_count_opt, rows,
               n_kv_heads, head_dim, d_kpool, d_vpool, d_scales, num_pages, d_error_opt, cuda_stream);
}

}  // extern "C"
