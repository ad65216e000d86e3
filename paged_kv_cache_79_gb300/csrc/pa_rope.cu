// Rotary positions: queries and keys turned by their tokens' positions, the keys and
// values written through the slot map into the paged cache in the same launch.
//
// Pair i of a head (elements i and i + half, or 2i and 2i + 1; half = rotary_dim / 2) of a
// token at position p turns by the angle p * theta_i:
//     (a, b) -> amplitude * (a cos - b sin, b cos + a sin)
// theta_i comes as F_i, the turns of a full circle per position in units of 2^-64, so
// p * F_i modulo 2^64, one 64-bit product, is the fraction of a turn exactly: positions far
// beyond 2^24, where a 32-bit p * theta has lost the angle, cost nothing extra.
//
// Bound by bytes: each of q, k, v is read once and written once.  A CTA takes a run of
// units, 32 bytes of a head each: for a rotated unit the 16-byte vectors that hold both
// elements of its pairs.  It first computes the cosines and sines of its tokens into shared
// memory, once for all heads of a token.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pagedkv {

namespace {

constexpr int kRopeThreads = 256;
// Units per thread: one where the grid would not fill the GPU eight CTAs deep twice over (64
// tokens of 64/8 heads: 2.7 us), else three (32768 tokens of 32/8 heads bf16: 150.9 us with
// one, 148.6 with two, 142.4 with three, 147.8 with four; 5660 GB/s, 83% of the copy's rate).
constexpr int kManyUnits = 3;

// Elements of a 16-byte vector as fp32, and back.
template <typename T>
struct Vec {
    static constexpr int kN = 16 / (int)sizeof(T);
    static __device__ __forceinline__ void unpack(const uint4 &x, float (&f)[kN])
    {
        const T *t = reinterpret_cast<const T *>(&x);
#pragma unroll
        for (int i = 0; i < kN; ++i)
            f[i] = static_cast<float>(t[i]);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[kN])
    {
        uint4 x;
        T *t = reinterpret_cast<T *>(&x);
#pragma unroll
        for (int i = 0; i < kN; ++i)
            t[i] = dev::from_float<T>(f[i]);
        return x;
    }
};

// kUnits: units per thread.
template <typename T, int kUnits>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int kN = Vec<T>::kN;
    extern __shared__ float2 table[];  // [token of the CTA][pair]: cosine, sine
    dev::grid_dependency_wait();
    dev::grid_launch_dependents();
    const int tid = threadIdx.x;
    const int per_head = p.head_dim / (2 * kN);  // units
    const int per_token = p.units_per_token;
    const long long w0 = (long long)blockIdx.x * (kRopeThreads * kUnits);
    const int t0 = (int)(w0 / per_token);
    const int off0 = (int)(w0 - (long long)t0 * per_token);
    const int tokens = min(p.num_tokens - t0, (off0 + kRopeThreads * kUnits - 1) / per_token + 1);

    // The loads do not wait for the table.
    uint4 x[kUnits][2];
    uint4 *dst[kUnits];
    int at[kUnits], second[kUnits];  // row of the table (-1: a copy), distance of the second vector
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        dst[u] = nullptr;
        const int l = off0 + tid + u * kRopeThreads;
        const int tl = l / per_token;
        if (tl >= tokens)
            continue;
        const int r = l - tl * per_token, head = r / per_head, i = r - head * per_head;
        const long long t = t0 + tl;
        const bool rotated = i * kN < p.half && head < p.num_q_heads + p.num_kv_heads;
        // the first vector of the unit, and the second's distance
        const int first = rotated && !p.interleaved ? i : 2 * i;
        second[u] = rotated && !p.interleaved ? p.half / kN : 1;
        at[u] = rotated ? tl * p.half + i * kN : -1;
        const T *src;
        T *d;
        if (head < p.num_q_heads) {
            src = static_cast<const T *>(p.q) + t * p.q_stride + head * p.head_dim;
            d = static_cast<T *>(p.q_out) + t * p.q_out_stride + head * p.head_dim;
        } else {
            const bool is_k = head < p.num_q_heads + p.num_kv_heads;
            const int h = head - p.num_q_heads - (is_k ? 0 : p.num_kv_heads);
            src = is_k ? static_cast<const T *>(p.k) + t * p.k_stride
                       : static_cast<const T *>(p.v) + t * p.v_stride;
            long long row = t;
            if (p.slots) {
                row = p.slots[t];
                if (row < 0 || row >= p.num_slots)
                    continue;
            }
            src += h * p.head_dim;
            d = static_cast<T *>(is_k ? p.k_out : p.v_out) + row * p.k_out_stride + h * p.head_dim;
        }
        const uint4 *s4 = reinterpret_cast<const uint4 *>(src) + first;
        dst[u] = reinterpret_cast<uint4 *>(d) + first;
        x[u][0] = s4[0];
        x[u][1] = s4[second[u]];
    }

    for (int i = tid; i < tokens * p.half; i += kRopeThreads) {
        const int tl = i / p.half;
        const unsigned long long turn =
            (unsigned long long)(long long)p.positions[t0 + tl] * p.freqs[i - tl * p.half];
        // rounded to 32 bits: half turns in units of 2^-31
        const int half_turns = (int)(unsigned int)((turn + 0x80000000ull) >> 32);
        float s, c;
        sincospif((float)half_turns * 0x1p-31f, &s, &c);
        table[i] = make_float2(c * p.amplitude, s * p.amplitude);
    }
    __syncthreads();

#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        if (!dst[u])
            continue;
        if (at[u] >= 0) {
            float a[kN], b[kN];
            Vec<T>::unpack(x[u][0], a);
            Vec<T>::unpack(x[u][1], b);
            const float2 *cs = table + at[u];
            if (p.interleaved) {
#pragma unroll
                for (int i = 0; i < kN; i += 2) {
                    const float2 f = cs[i / 2], g = cs[i / 2 + kN / 2];
                    const float a0 = a[i], b0 = b[i];
                    a[i] = a0 * f.x - a[i + 1] * f.y;
                    a[i + 1] = a[i + 1] * f.x + a0 * f.y;
                    b[i] = b0 * g.x - b[i + 1] * g.y;
                    b[i + 1] = b[i + 1] * g.x + b0 * g.y;
                }
            } else {
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    const float2 f = cs[i];
                    const float a0 = a[i];
                    a[i] = a0 * f.x - b[i] * f.y;
                    b[i] = b[i] * f.x + a0 * f.y;
                }
            }
            x[u][0] = Vec<T>::pack(a);
            x[u][1] = Vec<T>::pack(b);
        }
        dst[u][0] = x[u][0];
        dst[u][second[u]] = x[u][1];
    }
}

template <typename T, int kUnits>
cudaError_t launch_rope_units(const RopeParams &p, long long units, cudaStream_t stream)
{
    const int per_cta = kRopeThreads * kUnits;
    const long long ctas = (units + per_cta - 1) / per_cta;
    if (ctas > 0x7fffffffll)
        return cudaErrorInvalidValue;
    const int tokens = (int)std::fmin((double)p.num_tokens, (double)((per_cta - 1) / p.units_per_token + 2));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kRopeThreads);
    cfg.dynamicSmemBytes = (size_t)tokens * p.half * sizeof(float2);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rope_kernel<T, kUnits>, p);
}

template <typename T>
cudaError_t launch_rope_type(RopeParams p, int sms, cudaStream_t stream)
{
    const int per_head = p.head_dim / (2 * Vec<T>::kN);
    p.units_per_token = (p.num_q_heads + p.num_kv_heads * (p.v ? 2 : 1)) * per_head;
    const long long units = (long long)p.num_tokens * p.units_per_token;
    if (units >= (long long)sms * 8 * kRopeThreads * 2)
        return launch_rope_units<T, kManyUnits>(p, units, stream);
    return launch_rope_units<T, 1>(p, units, stream);
}

pa_status rope_impl(RopeParams &p, int block_size, int num_blocks, int dtype, void *stream)
{
    if (p.num_tokens == 0)
        return PA_OK;
    if (!p.q_out || !p.q || !p.k_out || !p.k || !p.positions || !p.freqs)
        return PA_ERR_INVALID;
    const int rotary_dim = 2 * p.half;
    if (p.num_tokens < 0 || p.num_q_heads <= 0 || p.num_kv_heads <= 0 || p.head_dim <= 0 ||
        block_size <= 0 || num_blocks <= 0 || rotary_dim <= 0 || rotary_dim > p.head_dim ||
        !std::isfinite(p.amplitude))
        return PA_ERR_INVALID;
    if (!dtype_ok(dtype) || (p.head_dim != 64 && p.head_dim != 128) || rotary_dim % 16 != 0)
        return PA_ERR_UNSUPPORTED;
    const long long q_row = (long long)p.num_q_heads * p.head_dim, k_row = (long long)p.num_kv_heads * p.head_dim;
    if (q_row + 2 * k_row > (1ll << 24))
        return PA_ERR_UNSUPPORTED;
    const int per_vec = dtype == PA_F32 ? 4 : 8;
    // (one token has no next row, so its strides may be anything)
    if (p.num_tokens > 1) {
        for (const long long s : {p.q_stride, p.q_out_stride, p.k_stride, p.k_out_stride, p.v ? p.v_stride : 0})
            if (s % per_vec != 0)
                return PA_ERR_INVALID;
        if (p.q_stride < q_row || p.q_out_stride < q_row || p.k_stride < k_row || p.k_out_stride < k_row ||
            (p.v && p.v_stride < k_row))
            return PA_ERR_INVALID;
    }
    for (const void *ptr : {(const void *)p.q, (const void *)p.q_out, (const void *)p.k, (const void *)p.k_out,
                            p.v, (const void *)p.v_out})
        if (!aligned(ptr, 16))
            return PA_ERR_INVALID;
    if (!aligned(p.positions, 4) || !aligned(p.freqs, 8) || !aligned(p.slots, 8))
        return PA_ERR_INVALID;
    if ((long long)num_blocks * block_size >= (1ll << 31))
        return PA_ERR_INVALID;
    p.num_slots = (long long)num_blocks * block_size;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess)
        return cuda_fail(e);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int sms = sm_count(device);
    e = dtype == PA_F32   ? launch_rope_type<float>(p, sms, st)
        : dtype == PA_F16 ? launch_rope_type<__half>(p, sms, st)
                          : launch_rope_type<__nv_bfloat16>(p, sms, st);
    return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

}  // namespace

}  // namespace pagedkv

using namespace pagedkv;

extern "C" {

pa_status pa_rope(void *q_out, long long q_out_stride, const void *q, long long q_stride, void *k_out,
                  long long k_out_stride, const void *k, long long k_stride, const int32_t *positions,
                  const int64_t *freqs, int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                  int rotary_dim, int interleaved, float amplitude, pa_dtype dtype, void *stream)
{
    if (rotary_dim < 0 || rotary_dim % 2 != 0)
        return PA_ERR_INVALID;
    RopeParams p = {};
    p.q_out = q_out;
    p.q = q;
    p.k_out = k_out;
    p.k = k;
    p.q_out_stride = q_out_stride;
    p.q_stride = q_stride;
    p.k_out_stride = k_out_stride;
    p.k_stride = k_stride;
    p.positions = positions;
    p.freqs = reinterpret_cast<const unsigned long long *>(freqs);
    p.num_tokens = num_tokens;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.half = rotary_dim / 2;
    p.interleaved = interleaved != 0;
    p.amplitude = amplitude;
    return rope_impl(p, 1, 1, dtype, stream);
}

pa_status pa_rope_append(void *q_out, long long q_out_stride, const void *q, long long q_stride,
                         const void *k, long long k_stride, const void *v, long long v_stride,
                         void *k_cache, void *v_cache, const int32_t *positions,
                         const int64_t *slot_mapping, const int64_t *freqs, int num_tokens,
                         int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim, int interleaved,
                         float amplitude, int block_size, int num_blocks, pa_dtype dtype, void *stream)
{
    if (num_tokens == 0)
        return PA_OK;
    if (!v || !v_cache || !slot_mapping || rotary_dim < 0 || rotary_dim % 2 != 0)
        return PA_ERR_INVALID;
    RopeParams p = {};
    p.q_out = q_out;
    p.q = q;
    p.k_out = k_cache;
    p.k = k;
    p.v_out = v_cache;
    p.v = v;
    p.q_out_stride = q_out_stride;
    p.q_stride = q_stride;
    p.k_out_stride = (long long)num_kv_heads * head_dim;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.positions = positions;
    p.slots = slot_mapping;
    p.freqs = reinterpret_cast<const unsigned long long *>(freqs);
    p.num_tokens = num_tokens;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.half = rotary_dim / 2;
    p.interleaved = interleaved != 0;
    p.amplitude = amplitude;
    return rope_impl(p, block_size, num_blocks, dtype, stream);
}

pa_status pa_rope_frequencies(int64_t *freqs, float *amplitude, int rotary_dim, double base,
                              pa_rope_scaling scaling, double factor, double original_len, double low,
                              double high)
{
    if (!freqs || !amplitude || rotary_dim <= 0 || rotary_dim % 2 != 0 || !(base > 1.0) ||
        !std::isfinite(base))
        return PA_ERR_INVALID;
    if ((int)scaling < PA_ROPE_NONE || (int)scaling > PA_ROPE_YARN)
        return PA_ERR_UNSUPPORTED;
    const bool by_length = scaling == PA_ROPE_BANDS || scaling == PA_ROPE_YARN;
    if (scaling != PA_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
        return PA_ERR_INVALID;
    if (by_length && (!(original_len > 0.0) || !std::isfinite(original_len) || !(low > 0.0) ||
                      !(high > low) || !std::isfinite(high)))
        return PA_ERR_INVALID;
    const double pi = 3.14159265358979323846;
    const int half = rotary_dim / 2;
    if (scaling == PA_ROPE_NTK)
        base *= std::pow(factor, rotary_dim > 2 ? (double)rotary_dim / (rotary_dim - 2) : 1.0);
    // yarn: the pairs' indices at which `high` and `low` turns fit the original length
    double first = 0.0, last = 0.0;
    if (scaling == PA_ROPE_YARN) {
        first = std::fmax(std::floor(rotary_dim * std::log(original_len / (high * 2 * pi)) / (2 * std::log(base))), 0.0);
        last = std::fmin(std::ceil(rotary_dim * std::log(original_len / (low * 2 * pi)) / (2 * std::log(base))),
                         (double)rotary_dim - 1);
    }
    for (int i = 0; i < half; ++i) {
        const double f = std::pow(base, -2.0 * i / rotary_dim);
        double keep = 1.0;  // the share of the unscaled angle
        if (scaling == PA_ROPE_LINEAR)
            keep = 0.0;
        else if (scaling == PA_ROPE_BANDS)
            keep = (original_len * f / (2 * pi) - low) / (high - low);
        else if (scaling == PA_ROPE_YARN)
            keep = 1.0 - (i - first) / std::fmax(last - first, 0.001);
        keep = std::fmin(std::fmax(keep, 0.0), 1.0);
        const double g = scaling == PA_ROPE_NONE || scaling == PA_ROPE_NTK ? f : f / factor * (1.0 - keep) + f * keep;
        double turns = g / (2 * pi);
        turns -= std::floor(turns);
        const double units = std::nearbyint(std::ldexp(turns, 64));
        freqs[i] = units >= 18446744073709551616.0 ? 0 : (int64_t)(uint64_t)units;
    }
    *amplitude = scaling == PA_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
    return PA_OK;
}

}  // extern "C"
