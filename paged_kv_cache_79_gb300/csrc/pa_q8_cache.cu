// Append to the 8-bit paged cache: new K and V rows become e4m3 codes under the scale
// of their (block, kv head).
//
// For every block that gets new rows, and each of K and V of each kv head:
//     need = the smallest power of two with max |x| <= 448 need over the new rows
//     s    = need when the block's first row is among them (the block starts anew),
//            else max(old s, need)
//     code = e4m3(x / s); where s grew, the block's other rows become
//            e4m3(code * old / s)
// 448 is e4m3's largest value.  With powers of two, x / s is exact, so a code is its
// value rounded once, and rounding again loses nothing but what falls below e4m3's
// smallest normal number: e4m3 keeps its 4 significant bits over 2^-6 .. 448 wherever
// the maximum lies, so a scale that fits the maximum exactly would gain nothing.
//
// One warp has one (block, kv head, K or V): its rows' maximum, the old scale, the codes
// and, where the scale grew, the rest of the tile are read and written by that warp
// alone, so nothing is exchanged.  Bound by the bytes of the rows and codes for prompts,
// by two dependent reads (lengths and table, then rows and scale) for single tokens: 16
// prompts of 40 heads take 78.4 us, 97% of the measured copy's rate; 256 single tokens 3.2.
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pagedkv {

namespace {

constexpr int kAppendWarps = 8;
constexpr int kChunk = 32;  // tokens a CTA looks through for the first rows of blocks

// A run of new rows in one block.
struct Run {
    int token;  // first row of k and v
    int rows;
    int block;
    int off;    // first row in the block
};

// The run that starts at token t, or rows = 0 when none does.
__device__ __forceinline__ Run run_at(const Q8AppendParams &p, int t, int s, int start, int n)
{
    Run r = {t, 0, 0, 0};
    const long long pos = (long long)p.context_lens[s] - n + (t - start);
    if (pos < 0 || pos >= (long long)p.max_blocks * p.block_size)
        return r;
    r.off = (int)(pos % p.block_size);
    if (r.off != 0 && t != start)
        return r;  // a row behind the first of its block's
    r.block = p.block_tables[(size_t)s * p.max_blocks + pos / p.block_size];
    if (r.block < 0 || r.block >= p.num_blocks)
        return r;
    r.rows = min(min(p.block_size - r.off, n - (t - start)), p.num_tokens - t);
    return r;
}

__device__ __forceinline__ void widen(float (&x)[8], const uint4 &w, const __half *)
{
    const __half2 *h = reinterpret_cast<const __half2 *>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(h[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void widen(float (&x)[8], const uint4 &w, const __nv_bfloat16 *)
{
    const uint32_t *u = reinterpret_cast<const uint32_t *>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void widen(float (&x)[4], const uint4 &w, const float *)
{
    x[0] = __uint_as_float(w.x);
    x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z);
    x[3] = __uint_as_float(w.w);
}

// Largest |x| of the 16 bytes as the bits of its type, without the sign: in this order
// infinities, then NaN, lie above every finite value.
__device__ __forceinline__ uint32_t abs_max_bits(uint32_t m, const uint4 &w, const float *)
{
    m = max(m, w.x & 0x7fffffffu);
    m = max(m, w.y & 0x7fffffffu);
    m = max(m, w.z & 0x7fffffffu);
    return max(m, w.w & 0x7fffffffu);
}
template <typename T>  // two 16-bit values at a time
__device__ __forceinline__ uint32_t abs_max_bits(uint32_t m, const uint4 &w, const T *)
{
    m = __vmaxu2(m, w.x & 0x7fff7fffu);
    m = __vmaxu2(m, w.y & 0x7fff7fffu);
    m = __vmaxu2(m, w.z & 0x7fff7fffu);
    return __vmaxu2(m, w.w & 0x7fff7fffu);
}

// A warp's maximum of those bits as fp32 (infinite or NaN when some value is).
__device__ __forceinline__ float warp_abs_max(uint32_t m, const float *)
{
    return __uint_as_float(__reduce_max_sync(0xffffffffu, m));
}
__device__ __forceinline__ float warp_abs_max(uint32_t m, const __nv_bfloat16 *)
{
    return __uint_as_float(__reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16)) << 16);
}
__device__ __forceinline__ float warp_abs_max(uint32_t m, const __half *)
{
    return __half2float(__ushort_as_half(
        (unsigned short)__reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16))));
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d)
{
    return dev::f32x2_to_e4m3x2(a, b) | (dev::f32x2_to_e4m3x2(c, d) << 16);
}

// x / s with NaN for values that are not finite (the conversion would make infinities
// +-448).
__device__ __forceinline__ float quotient(float x, float s)
{
    return finite(x) ? x / s : __uint_as_float(0x7fffffffu);
}

// Four codes times `ratio`, rounded again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio)
{
    uint32_t h0, h1;
    dev::e4m3x4_to_f16x4(w, h0, h1);
    const float2 f0 = __half22float2(*reinterpret_cast<const __half2 *>(&h0));
    const float2 f1 = __half22float2(*reinterpret_cast<const __half2 *>(&h1));
    return encode4(f0.x * ratio, f0.y * ratio, f1.x * ratio, f1.y * ratio);
}

constexpr int hold(int rows, int elem_bytes, int head_dim)  // loads of 16 bytes that a lane keeps
{
    return rows * head_dim * elem_bytes / 512 < 16 ? rows * head_dim * elem_bytes / 512 : 16;
}

// kRows: rows of a run whose loads are kept in registers, and all in flight at once; a
// longer run's other rows are read twice.  Up to eight loads per lane leave room for four
// CTAs on an SM (16 prompts, 40 heads, 16-row blocks: 92 us with two, 81 with three, 79
// with four).
template <typename T, int D, int BS, int kRows>
__global__ void __launch_bounds__(32 * kAppendWarps, hold(kRows, sizeof(T), D) <= 8 ? 4 : 2)
    q8_append_kernel(const __grid_constant__ Q8AppendParams p)
{
    constexpr int E = 16 / (int)sizeof(T);    // elements of a 16-byte load
    constexpr int LR = D / E;                 // lanes on one row
    constexpr int RP = 32 / LR;               // rows a warp loads at once
    constexpr int kPasses = BS / RP;
    constexpr int kHold = hold(kRows, sizeof(T), D);
    static_assert(kHold >= 1, "a load at least");
    __shared__ Run runs[kChunk];
    __shared__ int num_runs;
    dev::grid_dependency_wait();  // lengths, tables, rows and cache may come from the previous kernel
    dev::grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) {
        const int t0 = blockIdx.x * kChunk, t = t0 + lane;
        Run r = {t, 0, 0, 0};
        if (p.query_start) {
            // a decode step's rows: one per sequence, so that row t is sequence t's; a look
            // at those entries saves the search
            const int at = min(t, p.num_seqs), next = min(t + 1, p.num_seqs);
            int start = p.query_start[at], end = p.query_start[next], s = t;
            if (!__all_sync(0xffffffffu, t >= p.num_tokens || (t < p.num_seqs && start == t && end == t + 1))) {
                s = dev::find_sequence(p.query_start, p.num_seqs, t0, lane);
                if (s >= 0 && s < p.num_seqs) {
                    start = p.query_start[s];
                    end = p.query_start[s + 1];
                }
            }
            if (t < p.num_tokens && s >= 0 && s < p.num_seqs)
                r = run_at(p, t, s, start, end - start);
        } else if (t < p.num_tokens && t < p.num_seqs) {
            r = run_at(p, t, t, t, 1);
        }
        const unsigned has = __ballot_sync(0xffffffffu, r.rows > 0);
        if (r.rows > 0)
            runs[__popc(has & ((1u << lane) - 1u))] = r;
        if (lane == 0)
            num_runs = __popc(has);
    }
    __syncthreads();
    const int tiles = 2 * p.num_kv_heads;  // (kv head, K or V)
    const int tasks = num_runs * tiles;
    for (int task = blockIdx.y * kAppendWarps + warp; task < tasks; task += gridDim.y * kAppendWarps) {
        const Run r = runs[task / tiles];
        const int tile = task % tiles;
        const T *src = reinterpret_cast<const T *>((tile & 1) ? p.v : p.k) +
                       ((size_t)r.token * p.num_kv_heads + (tile >> 1)) * D + (lane % LR) * E;
        const size_t row_stride = (size_t)p.num_kv_heads * D;
        uint8_t *const block = p.cache + (size_t)r.block * p.block_bytes;
        uint8_t *const codes = block + (size_t)tile * (BS * D);
        float *const scale = reinterpret_cast<float *>(block + p.scales) + tile;
        const float old = r.off == 0 ? 0.f : *scale;
        const int row0 = lane / LR;  // this lane's rows: row0, row0 + RP, ...
        auto load = [&](int i) {
            const int row = i * RP + row0;
            return row < r.rows ? __ldcg(reinterpret_cast<const uint4 *>(src + row * row_stride))
                                : make_uint4(0, 0, 0, 0);
        };

        uint4 w[kHold];
#pragma unroll
        for (int i = 0; i < kHold; ++i)
            w[i] = load(i);
        uint32_t bits = 0;
#pragma unroll
        for (int i = 0; i < kHold; ++i)
            bits = abs_max_bits(bits, w[i], src);
        for (int i = kHold; i < kPasses && i * RP < r.rows; ++i)
            bits = abs_max_bits(bits, load(i), src);
        float top = warp_abs_max(bits, src);
        float x[E];
        const bool odd = !finite(top);  // some value is infinite or NaN: leave those out
        if (odd) {
            top = 0.f;
            for (int i = 0; i < kPasses && i * RP < r.rows; ++i) {
                widen(x, load(i), src);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    top = finite(x[e]) ? fmaxf(top, fabsf(x[e])) : top;
            }
            top = dev::warp_max(top);
        }
        // 448 = 1.75 * 2^8: the exponent of top / 448, one more where top's mantissa
        // passes 1.75's; at least the smallest normal scale
        const int e2 = max((int)((__float_as_uint(top) + 0x1fffffu) >> 23) - 8, 1);
        const float need = __uint_as_float((uint32_t)e2 << 23);
        const float s = fmaxf(old, need);
        auto put = [&](int i) {
            const int row = i * RP + row0;
            if (row < r.rows) {
                uint8_t *dst = codes + (size_t)(r.off + row) * D + (lane % LR) * E;
                const uint32_t c0 = encode4(x[0], x[1], x[2], x[3]);
                if constexpr (E == 8)
                    *reinterpret_cast<uint2 *>(dst) = make_uint2(c0, encode4(x[4], x[5], x[6], x[7]));
                else
                    *reinterpret_cast<uint32_t *>(dst) = c0;
            }
        };
        if (!odd && (__float_as_uint(s) & 0x7fffffu) == 0) {
            const float inv = 1.f / s;  // exact: a power of two
#pragma unroll
            for (int i = 0; i < kHold; ++i) {
                widen(x, w[i], src);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    x[e] *= inv;
                put(i);
            }
            for (int i = kHold; i < kPasses && i * RP < r.rows; ++i) {
                widen(x, load(i), src);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    x[e] *= inv;
                put(i);
            }
        } else {
            // values that are not finite, or a scale of the caller's own
            for (int i = 0; i < kPasses && i * RP < r.rows; ++i) {
                widen(x, load(i), src);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    x[e] = quotient(x[e], s);
                put(i);
            }
        }
        if (r.off != 0 && s > old) {
            const float ratio = old / s;
            for (int v = lane; v < BS * D / 16; v += 32) {
                const int row = v * 16 / D;
                if (row >= r.off && row < r.off + r.rows)
                    continue;
                uint4 q = reinterpret_cast<const uint4 *>(codes)[v];
                q.x = rescale4(q.x, ratio);
                q.y = rescale4(q.y, ratio);
                q.z = rescale4(q.z, ratio);
                q.w = rescale4(q.w, ratio);
                reinterpret_cast<uint4 *>(codes)[v] = q;
            }
        }
        if (lane == 0 && (r.off == 0 || s != old))
            *scale = s;
    }
}

template <typename T, int D, int BS>
cudaError_t launch(const Q8AppendParams &p, int sms, cudaStream_t stream)
{
    // Short runs (up to four rows per sequence on average, as in a decode step) take the
    // variant that keeps four rows: more CTAs fit an SM, and a step's tiles all run at
    // once (256 single tokens, 8 heads, 32-row blocks: 3.2 us against 6.1).
    const bool few = p.num_tokens <= 4ll * p.num_seqs;
    // CTAs over the chunks, then over a chunk's tiles: at most one tile per warp for the
    // number of blocks a chunk can be expected to touch, and no more than twenty CTAs per
    // SM in all, so that long prompts' CTAs find their sequences once for several tiles
    // each (16 prompts, 40 heads: 82.4, 79.2 and 78.4 us with 6, 12 and 20).
    const long long chunks = ((long long)p.num_tokens + kChunk - 1) / kChunk;
    const long long runs = p.query_start ? ((long long)p.num_tokens + BS - 1) / BS + p.num_seqs : p.num_tokens;
    const long long per_chunk = ((runs < p.num_tokens ? runs : p.num_tokens) + chunks - 1) / chunks;
    const long long most = (per_chunk * 2 * p.num_kv_heads + kAppendWarps - 1) / kAppendWarps;
    const long long fill = (20ll * sms + chunks - 1) / chunks;
    const long long y = most < fill ? most : fill;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)chunks, (unsigned)(y < 65535 ? y : 65535));
    cfg.blockDim = dim3(32 * kAppendWarps);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return few ? cudaLaunchKernelEx(&cfg, q8_append_kernel<T, D, BS, 4>, p)
               : cudaLaunchKernelEx(&cfg, q8_append_kernel<T, D, BS, BS>, p);
}

template <typename T>
cudaError_t dispatch(const Q8AppendParams &p, int head_dim, int sms, cudaStream_t stream)
{
    if (head_dim == 128)
        return p.block_size == 16 ? launch<T, 128, 16>(p, sms, stream) : launch<T, 128, 32>(p, sms, stream);
    return p.block_size == 16 ? launch<T, 64, 16>(p, sms, stream) : launch<T, 64, 32>(p, sms, stream);
}

}  // namespace

cudaError_t launch_q8_append(const Q8AppendParams &p, int head_dim, pa_dtype dtype, int sms,
                             cudaStream_t stream)
{
    return dtype == PA_F32   ? dispatch<float>(p, head_dim, sms, stream)
           : dtype == PA_F16 ? dispatch<__half>(p, head_dim, sms, stream)
                             : dispatch<__nv_bfloat16>(p, head_dim, sms, stream);
}

}  // namespace pagedkv
