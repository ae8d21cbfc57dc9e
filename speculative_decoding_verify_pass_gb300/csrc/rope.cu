// Rotary positions of a call's rows.
//
// Pair i of a head, i < r/2, is turned by the angle pos * f_i:
//     u' = g (u cos - v sin),   v' = g (v cos + u sin)
// with (u, v) = (x[i], x[i + r/2]) or (x[2i], x[2i+1]).  The frequency is kept as a
// fraction of a circle per position in 64-bit fixed point, so that pos * f modulo
// one circle is one wrapping integer product, exact to pos * 2^-64 whatever the
// position; its upper 32 bits, as a signed fraction, go to sincospi.  (In fp32 the
// angle of position 500000 would be off by 2^-6.)
//
// Memory bounds it: x once in, once out.  A warp takes a row: it loads its first heads,
// finds the row's position, fills a table of cos and sin in shared memory, and then goes
// over the heads, a lane's pairs the same in each, so that their cos and sin stay in
// registers.  16001 rows of 40 heads of 128, 64 of them rotated, take 51.7 us (328 MB: 6.3
// TB/s); a CTA of 8 rows with one table that every piece looked up took 62.2.  2 heads
// in flight a lane: 1 took 57.5, 4 (and their registers) 61.1.  Few rows (at most 4 per
// SM) have 8 warps each, which all find the position and fill a table: 2.5 us for 8 rows.
#include <cuda_fp16.h>
#include <math.h>

#include "internal.h"
#include "spec.h"

namespace sv {
namespace {

constexpr int kWarps = 8;       // of a CTA
constexpr int kBatch = 2;       // heads that a lane has in flight

struct RopeParams {
    const void* x;
    void* out;
    long long x_stride, out_stride;             // elements
    const unsigned long long* turns;
    const int *row_start, *len, *pos;
    int nseq, rows, heads, hd, pairs;           // pairs: r/2
    int split;                                  // 2^split warps share a row
    float gain;
    int inverse, copy;                          // copy: elements behind the rotated part go to another buffer
};

template <class T>
__device__ __forceinline__ float up(T v);
template <>
__device__ __forceinline__ float up(float v) { return v; }
template <>
__device__ __forceinline__ float up(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float up(__half v) { return __half2float(v); }
template <class T>
__device__ __forceinline__ T down(float v);
template <>
__device__ __forceinline__ float down(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 down(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half down(float v) { return __float2half_rn(v); }

template <class T, int N>
struct alignas(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Piece {
    T v[N];
};

// The sequence that row r belongs to (-1: none), and where its rows end.  32 row
// starts a step: a warp needs two for 1024 sequences.
__device__ __forceinline__ int sequence(const int* start, int nseq, int r, int lane, int* end) {
    int lo = 0, n = nseq;                       // among the n sequences from lo on
    while (n > 1) {
        const int step = (n + 31) / 32, at = lo + lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, at < lo + n && start[at] <= r);
        const int k = below ? 31 - __clz(below) : 0;
        n = min(step, n - k * step);
        lo += k * step;
    }
    *end = start[lo + 1];
    return start[lo] <= r && r < *end ? lo : -1;
}

// What a lane takes at a time: VEC pairs of kBatch heads, as one piece (INTER) or two.
template <class T, int VEC, bool INTER>
struct Batch {
    static constexpr int N = INTER ? 2 * VEC : VEC, kPieces = INTER ? 1 : 2;
    Piece<T, N> a[kBatch][kPieces];
    __device__ __forceinline__ void load(const T* x, const RopeParams& p, int h, int step, int j) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (h + u * step < p.heads)
#pragma unroll
                for (int k = 0; k < kPieces; ++k)
                    a[u][k] = *reinterpret_cast<const Piece<T, N>*>(x + (h + u * step) * p.hd + (INTER ? 2 * j : j + k * p.pairs));
    }
    __device__ __forceinline__ void turn_store(T* out, const RopeParams& p, int h, int step, int j, const float2* cs) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (h + u * step >= p.heads) continue;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                T &v = a[u][0].v[INTER ? 2 * e : e], &w = a[u][kPieces - 1].v[INTER ? 2 * e + 1 : e];
                const float m = up(v), n = up(w);
                v = down<T>(m * cs[e].x - n * cs[e].y);
                w = down<T>(n * cs[e].x + m * cs[e].y);
            }
#pragma unroll
            for (int k = 0; k < kPieces; ++k)
                *reinterpret_cast<Piece<T, N>*>(out + (h + u * step) * p.hd + (INTER ? 2 * j : j + k * p.pairs)) = a[u][k];
        }
    }
};

template <class T, int VEC, bool INTER>
__global__ void __launch_bounds__(32 * kWarps) rope_kernel(const __grid_constant__ RopeParams p) {
    extern __shared__ float2 tables[];          // [warps][pairs] cos, sin
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = (int)(((long long)blockIdx.x * kWarps + warp) >> p.split), part = warp & ((1 << p.split) - 1);
    // lanes: pieces of VEC pairs, over as many heads as there are lanes for
    const int pieces = p.pairs / VEC, across = min(pieces, 32), heads = 32 / across;
    const int j0 = lane % across * VEC, step = heads << p.split;
    const int h0 = lane / across < heads ? part * heads + lane / across : p.heads;
    pdl_wait();
    pdl_launch_dependents();
    if (r >= p.rows) return;
    const T* x = static_cast<const T*>(p.x) + r * p.x_stride;
    T* out = static_cast<T*>(p.out) + r * p.out_stride;
    Batch<T, VEC, INTER> batch;
    batch.load(x, p, h0, step, j0);         // (also of a row that is no sequence's)
    long long t = 0;
    if (p.pos) {
        t = p.pos[r];
    } else {
        int end;
        const int q = sequence(p.row_start, p.nseq, r, lane, &end);
        if (q < 0) return;
        t = (long long)p.len[q] - (end - r);
    }
    float2* turn = tables + warp * p.pairs;
    for (int j = lane; j < p.pairs; j += 32) {
        const unsigned long long phase = (unsigned long long)t * p.turns[j];
        float s, c;
        sincospif((float)(int)(phase >> 32) * 0x1p-31f, &s, &c);
        turn[j] = make_float2(c * p.gain, (p.inverse ? -s : s) * p.gain);
    }
    __syncwarp();
#pragma unroll 1
    for (int j = j0; j < p.pairs; j += 32 * VEC) {
        float2 cs[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) cs[e] = turn[j + e];
#pragma unroll 1
        for (int h = h0; h < p.heads; h += kBatch * step) {
            if (j != j0 || h != h0) batch.load(x, p, h, step, j);
            batch.turn_store(out, p, h, step, j, cs);
        }
    }
    if (p.copy) {                               // the elements behind the rotated ones
        constexpr int N = 2 * VEC * sizeof(T) < 16 ? 2 * VEC : 16 / sizeof(T);   // rotary_dim is a multiple of 2 * VEC
        const int rest = (p.hd - 2 * p.pairs) / N, beside = min(rest, 32), rows = 32 / beside, stride = rows << p.split;
        if (lane / beside >= rows) return;
        for (int j = lane % beside; j < rest; j += 32) {
            const int at = 2 * p.pairs + j * N;
#pragma unroll 1
            for (int h = part * rows + lane / beside; h < p.heads; h += 2 * kBatch * stride) {
                Piece<T, N> a[2 * kBatch];
#pragma unroll
                for (int u = 0; u < 2 * kBatch; ++u)
                    if (h + u * stride < p.heads) a[u] = *reinterpret_cast<const Piece<T, N>*>(x + (h + u * stride) * p.hd + at);
#pragma unroll
                for (int u = 0; u < 2 * kBatch; ++u)
                    if (h + u * stride < p.heads) *reinterpret_cast<Piece<T, N>*>(out + (h + u * stride) * p.hd + at) = a[u];
            }
        }
    }
}

// Pairs a lane takes: 16 bytes' worth where the pairs allow it.
template <class T, bool INTER>
const void* variant(int pairs) {
    constexpr int kMost = 16 / sizeof(T) / (INTER ? 2 : 1), kSome = kMost / 2;
    return pairs % kMost == 0   ? (const void*)rope_kernel<T, kMost, INTER>
           : pairs % kSome == 0 ? (const void*)rope_kernel<T, kSome, INTER>
                                : (const void*)rope_kernel<T, 1, INTER>;
}
template <class T>
const void* variant(int pairs, bool inter) { return inter ? variant<T, true>(pairs) : variant<T, false>(pairs); }

spec_status bad(const char* msg) {
    set_last_error(msg);
    return SPEC_ERR_INVALID_ARG;
}

bool misaligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

}  // namespace
}  // namespace sv

extern "C" {

using namespace sv;

spec_status spec_rope_table(int32_t rotary_dim, double base, int32_t scaling, double factor, double low, double high,
                            int32_t context, uint64_t* out_turns, float* out_gain) {
    if (!out_turns || !out_gain) return bad("spec_rope_table: null pointer");
    if (rotary_dim < 2 || rotary_dim > SPEC_ROPE_MAX_DIM || rotary_dim % 2) return bad("spec_rope_table: rotary_dim must be even, 2..1024");
    if (!(base > 1.0) || !isfinite(base)) return bad("spec_rope_table: base must be above 1 and finite");
    if (scaling < SPEC_ROPE_PLAIN || scaling > SPEC_ROPE_PARTS) return bad("spec_rope_table: unknown scaling");
    if (scaling != SPEC_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor)))
        return bad("spec_rope_table: factor must be at least 1 and finite");
    if (scaling == SPEC_ROPE_BASE && rotary_dim < 4) return bad("spec_rope_table: a scaled base needs a rotary_dim above 2");
    const bool ramp = scaling == SPEC_ROPE_WAVELENGTH || scaling == SPEC_ROPE_PARTS;
    if (ramp && (!(low > 0.0) || !(high > low) || !isfinite(high) || context < 1))
        return bad("spec_rope_table: a ramp needs 0 < low < high and a context of at least 1");
    const double circle = 6.283185307179586476925286766559;
    double b = base, first = 0, last = 0;
    if (scaling == SPEC_ROPE_BASE) b = base * pow(factor, (double)rotary_dim / (rotary_dim - 2));
    if (scaling == SPEC_ROPE_PARTS) {           // the pairs that turn `high` and `low` times in the context
        first = floor(rotary_dim * log(context / (circle * high)) / (2 * log(base)));
        last = ceil(rotary_dim * log(context / (circle * low)) / (2 * log(base)));
        first = first < 0 ? 0 : first;
        last = last > rotary_dim - 1 ? rotary_dim - 1 : last;
    }
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = pow(b, -2.0 * i / rotary_dim), keep = 1.0;
        if (scaling == SPEC_ROPE_LINEAR) keep = 0.0;
        if (scaling == SPEC_ROPE_WAVELENGTH) keep = (context * f / circle - low) / (high - low);
        if (scaling == SPEC_ROPE_PARTS) keep = i >= last ? 0.0 : i <= first ? 1.0 : 1.0 - (i - first) / (last - first);
        keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
        if (keep < 1.0) f = keep * f + (1.0 - keep) * f / factor;
        out_turns[i] = (uint64_t)nearbyint(f / circle * 18446744073709551616.0);    // f <= 1: below 2^62
    }
    *out_gain = scaling == SPEC_ROPE_PARTS ? (float)(0.1 * log(factor) + 1.0) : 1.f;
    return SPEC_OK;
}

spec_status spec_rope(const void* d_x, int64_t x_stride, void* d_out, int64_t out_stride, int32_t type, int32_t rows,
                      int32_t heads, int32_t head_dim, int32_t rotary_dim, int32_t interleaved, int32_t inverse, float gain,
                      const uint64_t* d_turns, const int32_t* d_row_start_opt, const int32_t* d_len_opt, int32_t nseq,
                      const int32_t* d_pos_opt, void* cuda_stream) {
    if (type != SPEC_BF16 && type != SPEC_FP16 && type != SPEC_FP32) return bad("spec_rope: type must be bf16, fp16 or fp32");
    if (rows < 0) return bad("spec_rope: negative rows");
    if (heads < 1 || heads > 4096) return bad("spec_rope: heads must be in 1..4096");
    if (head_dim < 8 || head_dim > SPEC_ROPE_MAX_DIM || head_dim % 8) return bad("spec_rope: head_dim must be a multiple of 8, 8..1024");
    if (rotary_dim < 2 || rotary_dim > head_dim || rotary_dim % 2) return bad("spec_rope: rotary_dim must be even and at most head_dim");
    if (!isfinite(gain)) return bad("spec_rope: gain must be finite");
    const int64_t row = (int64_t)heads * head_dim, whole = type == SPEC_FP32 ? 4 : 8;
    if (x_stride < row || out_stride < row || x_stride % whole || out_stride % whole || x_stride >= (1ll << 38) || out_stride >= (1ll << 38))
        return bad("spec_rope: row strides must be multiples of 16 bytes, at least heads * head_dim and below 2^38");
    // (no lengths may be a null pointer)
    if (d_pos_opt ? d_row_start_opt || d_len_opt : !d_row_start_opt || (!d_len_opt && nseq != 0)) {
        if (rows) return bad("spec_rope: positions come from d_pos, or from d_row_start and d_len (one of the two)");
    }
    if (!d_pos_opt && (nseq < 0 || nseq > SPEC_MAX_SEQS)) return bad("spec_rope: nseq must be in 0..1024");
    if (rows == 0 || (!d_pos_opt && nseq == 0)) return SPEC_OK;
    if (!d_x || !d_out || !d_turns) return bad("spec_rope: null pointer");
    if (misaligned(d_x, 16) || misaligned(d_out, 16)) return bad("spec_rope: rows must be 16-byte aligned");
    if (misaligned(d_turns, 8)) return bad("spec_rope: d_turns is not 8-byte aligned");
    if (misaligned(d_row_start_opt, 4) || misaligned(d_len_opt, 4) || misaligned(d_pos_opt, 4))
        return bad("spec_rope: an int32 pointer is not 4-byte aligned");
    if (d_x == d_out && x_stride != out_stride) return bad("spec_rope: in place, both strides must be the same");
    const int sms = current_sms();
    if (!sms) {
        set_last_error("spec_rope: no current CUDA device");
        return SPEC_ERR_CUDA;
    }
    RopeParams p;
    p.x = d_x;
    p.out = d_out;
    p.x_stride = x_stride;
    p.out_stride = out_stride;
    p.turns = reinterpret_cast<const unsigned long long*>(d_turns);
    p.row_start = d_row_start_opt;
    p.len = d_len_opt;
    p.pos = d_pos_opt;
    p.nseq = nseq;
    p.rows = rows;
    p.heads = heads;
    p.hd = head_dim;
    p.pairs = rotary_dim / 2;
    p.gain = gain;
    p.inverse = inverse != 0;
    p.copy = d_x != d_out && rotary_dim < head_dim;
    p.split = rows <= 4 * sms ? 3 : 0;
    const void* fn = type == SPEC_BF16   ? variant<__nv_bfloat16>(p.pairs, interleaved != 0)
                     : type == SPEC_FP16 ? variant<__half>(p.pairs, interleaved != 0)
                                         : variant<float>(p.pairs, interleaved != 0);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((((int64_t)rows << p.split) + kWarps - 1) / kWarps));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = (size_t)kWarps * p.pairs * sizeof(float2);       // at most 32 KB
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

}  // extern "C"
