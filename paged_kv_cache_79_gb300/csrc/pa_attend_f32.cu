// pa_attend for fp32: mma.sync with each operand in two tf32 terms.
//
// Tensor cores take fp32 operands as tf32 (11 significant bits).  x = hi + lo, hi
// rounded to that, leaves a product as hi hi' + hi lo' + lo hi', off by 2^-22 of itself at most,
// accumulated in fp32: three instructions per product.  (tcgen05 takes both operands from shared memory or TMEM as
// they are, so the split would have to be written there first, four tiles for each one.)
//
// A CTA's four warps hold 16 rows each of a tile of 64 rows, and step through tiles of 32 keys
// in two buffers, the next one's copies in flight while this one is multiplied.  Scores
// stay in registers: the fragment that Q K^T leaves becomes P's when a step of 8 keys is taken
// in the order 0 2 4 6 1 3 5 7, which only means reading V's rows in that order.
//
// Tiles with values that two terms do not stand for (NaN, infinities, numbers next to the largest)
// are multiplied by fp32 FMAs: V's are looked for as a tile arrives, in the scores what is not
// finite gives them away.
//
// Measured: 7 ragged chunks of up to 700 tokens on up to 1003 keys, 39 / 3 heads of 64 dims: 212 us,
// 29 TFLOP/s (220 with every term guarded).  Bound by the splitting (every warp splits the K and V
// that it reads; with conversion instructions instead of integer ones 462 us) and by reads of
// shared memory.
#include "pa_attend.cuh"

namespace pagedkv {

namespace {

constexpr int kF32Threads = 128;
constexpr int kF32Rows = kF32TileRows;
constexpr int kF32Keys = 32;

// hi: x rounded to tf32's 11 bits; lo: the rest (the tensor core cuts its last bit, 2^-23 of x).
// Of NaN, an infinity or a number that rounds to one (kSplitEnd on), at least one term is NaN or
// infinite, so sums that it is in are neither right nor finite: such tiles are multiplied by FMAs
// instead.
constexpr uint32_t kSplitEnd = 0x7f7ff000u;  // bits of |x|
__device__ __forceinline__ void split(float x, uint32_t &hi, uint32_t &lo)
{
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}

__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
        " {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_3(float (&c)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4], float b0,
                                      float b1)
{
    uint32_t h0, l0, h1, l1;
    split(b0, h0, l0);
    split(b1, h1, l1);
    mma_tf32(c, al, h0, h1);
    mma_tf32(c, ah, l0, l1);
    mma_tf32(c, ah, h0, h1);
}

// 16 bytes to shared memory, or zeros where the source is not there (src_bytes 0).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}

template <int D>
struct SmemF32 {
    static constexpr int kStride = D + 4;  // floats; rows 4 banks apart
    static constexpr int kPStride = kF32Keys + 1;
    float q[kF32Rows * kStride];
    float k[2][kF32Keys * kStride];
    float v[2][kF32Keys * kStride];
    float p[kF32Rows * kPStride];  // a tile's probabilities, for products by FMAs
    long long scratch[kF32Threads / 32 + 4];
};

template <int D>
__global__ void __launch_bounds__(kF32Threads) attend_f32_kernel(const __grid_constant__ AttendParams p)
{
    using Walk = AttendWalk<kF32Keys>;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    SmemF32<D> &sm = *reinterpret_cast<SmemF32<D> *>(smem_raw);
    constexpr int kStride = SmemF32<D>::kStride;
    constexpr int kVecs = D / 4;
    dev::grid_dependency_wait();
    dev::grid_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c4 = lane & 3;
    Walk walk(p);
    if (!walk.begin<kF32Threads>(sm.scratch))
        return;
    do {
        int a, b;
        if (!walk.part(a, b))
            continue;
        const AttendItem &it = walk.it;
        const auto rows = Walk::rows_of(p, it);
        const int num = rows.tokens * p.heads_per_item;
        const int32_t *table = p.block_tables + (size_t)it.s * p.max_blocks;

        auto load_kv = [&](int tile, int buf) {
            for (int i = tid; i < kF32Keys * kVecs; i += kF32Threads) {
                const int r = i / kVecs, x = i % kVecs;
                const int key = tile * kF32Keys + r;
                const int id = key < it.seen ? table[key / p.block_size] : -1;
                const bool there = id >= 0 && id < p.num_blocks;
                const size_t at =
                    there ? (((size_t)id * p.block_size + key % p.block_size) * p.num_kv_heads + rows.kv) * D + x * 4 : 0;
                cp_async16_or_zero(dev::smem_addr(&sm.k[buf][r * kStride + x * 4]),
                                   static_cast<const float *>(p.k_cache) + at, there);
                cp_async16_or_zero(dev::smem_addr(&sm.v[buf][r * kStride + x * 4]),
                                   static_cast<const float *>(p.v_cache) + at, there);
            }
        };
        __syncthreads();  // the previous item's tiles have been read
        for (int i = tid; i < kF32Rows * kVecs; i += kF32Threads) {
            const int r = i / kVecs, x = i % kVecs;
            const int tok = r / p.heads_per_item, head = r - tok * p.heads_per_item;
            const bool there = r < num && head < rows.heads;
            const float *src = static_cast<const float *>(p.q) +
                               (there ? (rows.token0 + tok) * p.q_stride + (size_t)(rows.head0 + head) * D + x * 4 : 0);
            cp_async16_or_zero(dev::smem_addr(&sm.q[r * kStride + x * 4]), src, there);
        }
        if (b > a)
            load_kv(a, 0);
        dev::cp_async_commit();

        // this thread's rows: r0 = 16 warp + g, and r0 + 8
        int limit[2];  // keys that the row sees
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int tok = (16 * warp + g + 8 * h) / p.heads_per_item;
            const long long last = (long long)it.T - it.n + it.j * (long long)p.tokens_per_item + tok + 1;
            limit[h] = p.causal ? (int)min(max(last, 0ll), (long long)it.T) : it.T;
        }
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float o[D / 8][4] = {};
        for (int tile = a; tile < b; ++tile) {
            const int buf = (tile - a) & 1;
            dev::cp_async_wait_all();
            // values that no two terms stand for: each thread looks at what it copied itself
            uint32_t largest = 0;
            for (int i = tid; i < kF32Keys * kVecs; i += kF32Threads) {
                const uint4 x = *reinterpret_cast<const uint4 *>(&sm.v[buf][i / kVecs * kStride + i % kVecs * 4]);
                largest = max(max(largest, max(x.x << 1, x.y << 1)), max(x.z << 1, x.w << 1));
            }
            // this tile's copies are there, the other buffer has been read
            const bool by_fma = __syncthreads_or(largest >= kSplitEnd << 1);
            if (tile + 1 < b)
                load_kv(tile + 1, buf ^ 1);
            dev::cp_async_commit();
            float s[kF32Keys / 8][4] = {};
#pragma unroll
            for (int k0 = 0; k0 < D; k0 += 8) {
                uint32_t ah[4], al[4];
                const float *qr = &sm.q[(16 * warp + g) * kStride + k0 + c4];
                split(qr[0], ah[0], al[0]);
                split(qr[8 * kStride], ah[1], al[1]);
                split(qr[4], ah[2], al[2]);
                split(qr[8 * kStride + 4], ah[3], al[3]);
#pragma unroll
                for (int n = 0; n < kF32Keys / 8; ++n) {
                    const float *kr = &sm.k[buf][(8 * n + g) * kStride + k0 + c4];
                    mma_3(s[n], ah, al, kr[0], kr[4]);
                }
            }
            // NaN, infinities and numbers next to them in q or K, or a sum past fp32's range
            bool finite = true;
#pragma unroll
            for (int n = 0; n < kF32Keys / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    finite = finite && fabsf(s[n][e]) < INFINITY;
            if (!finite) {
#pragma unroll
                for (int n = 0; n < kF32Keys / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[n][e] = 0.f;
#pragma unroll 1
                for (int k = 0; k < D; ++k) {
                    const float *qr = &sm.q[(16 * warp + g) * kStride + k], *kr = &sm.k[buf][2 * c4 * kStride + k];
                    const float q0 = qr[0], q1 = qr[8 * kStride];
#pragma unroll
                    for (int n = 0; n < kF32Keys / 8; ++n) {
                        const float k0 = kr[8 * n * kStride], k1 = kr[(8 * n + 1) * kStride];
                        s[n][0] = fmaf(q0, k0, s[n][0]);
                        s[n][1] = fmaf(q0, k1, s[n][1]);
                        s[n][2] = fmaf(q1, k0, s[n][2]);
                        s[n][3] = fmaf(q1, k1, s[n][3]);
                    }
                }
            }
            __syncwarp();
            const int key0 = tile * kF32Keys + 2 * c4;
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < kF32Keys / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool seen = key0 + 8 * n + (e & 1) < limit[e >> 1];
                    s[n][e] = seen ? s[n][e] * p.scale_log2 : -INFINITY;
                    // (fmaxf passes a NaN over; the sum does not)
                    top[e >> 1] = fmaxf(top[e >> 1], s[n][e]);
                }
            float scale[2], base[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
                top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
                const float now = fmaxf(m[h], top[h]);
                base[h] = now == -INFINITY ? 0.f : now;
                scale[h] = exp2f(m[h] - base[h]);
                m[h] = now;
                l[h] *= scale[h];
            }
            uint32_t ah[kF32Keys / 8][4], al[kF32Keys / 8][4];
#pragma unroll
            for (int n = 0; n < kF32Keys / 8; ++n) {
                float e[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    e[i] = exp2f(s[n][i] - base[i >> 1]);
                    l[i >> 1] += e[i];
                }
                // keys 2 c4 and 2 c4 + 1 of the step stand at its places c4 and c4 + 4
                split(e[0], ah[n][0], al[n][0]);
                split(e[2], ah[n][1], al[n][1]);
                split(e[1], ah[n][2], al[n][2]);
                split(e[3], ah[n][3], al[n][3]);
            }
            if (by_fma) {
                float *const pr = &sm.p[16 * warp * SmemF32<D>::kPStride];
#pragma unroll
                for (int n = 0; n < kF32Keys / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = e == 0 ? 0 : e == 1 ? 2 : e == 2 ? 1 : 3;  // (the order of the splits)
                        pr[(g + 8 * (e >> 1)) * SmemF32<D>::kPStride + 8 * n + 2 * c4 + (e & 1)] =
                            __uint_as_float(ah[n][i]) + __uint_as_float(al[n][i]);
                    }
                __syncwarp();
#pragma unroll
                for (int d = 0; d < D / 8; ++d) {
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                    for (int k = 0; k < kF32Keys; ++k) {
                        const float *vr = &sm.v[buf][k * kStride + 8 * d + 2 * c4];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            // (a hidden key's value may be anything)
                            if (tile * kF32Keys + k >= limit[h])
                                continue;
                            const float w = pr[(g + 8 * h) * SmemF32<D>::kPStride + k];
                            c[2 * h] = fmaf(w, vr[0], c[2 * h]);
                            c[2 * h + 1] = fmaf(w, vr[1], c[2 * h + 1]);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[d][e] = fmaf(o[d][e], scale[e >> 1], c[e]);
                }
                __syncwarp();  // the probabilities have been read
                continue;
            }
            // The tile's share of the output is summed by itself: the tensor core's additions cut
            // low bits off, which over a long context leans one way; the addition here rounds.
#pragma unroll
            for (int d = 0; d < D / 8; ++d) {
                float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int n = 0; n < kF32Keys / 8; ++n) {
                    const float *vr = &sm.v[buf][(8 * n + 2 * c4) * kStride + 8 * d + g];
                    mma_3(c, ah[n], al[n], vr[0], vr[kStride]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[d][e] = fmaf(o[d][e], scale[e >> 1], c[e]);
            }
        }
        dev::cp_async_wait_all();
        const bool whole = a == 0 && b == it.tiles;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            const int r = 16 * warp + g + 8 * h;
            const int tok = r / p.heads_per_item, head = r - tok * p.heads_per_item;
            if (r >= num || head >= rows.heads)
                continue;
            if (whole) {
                const size_t row = (size_t)(rows.token0 + tok) * p.num_q_heads + rows.head0 + head;
                const float inv = l[h] == 0.f ? 0.f : 1.f / l[h];
                float *dst = static_cast<float *>(p.out) + row * D + 2 * c4;
#pragma unroll
                for (int d = 0; d < D / 8; ++d)
                    *reinterpret_cast<float2 *>(dst + 8 * d) = make_float2(o[d][2 * h] * inv, o[d][2 * h + 1] * inv);
                if (p.lse && c4 == 0)
                    p.lse[row] = attend_lse<float>(m[h], l[h]);
            } else {
                const size_t row = attend_part_row(p, blockIdx.x, a > 0 ? 0 : 1) + r;
                if (c4 == 0)
                    p.part_ml[row] = make_float2(m[h], l[h]);
                float *dst = p.part_o + row * D + 2 * c4;
#pragma unroll
                for (int d = 0; d < D / 8; ++d)
                    *reinterpret_cast<float2 *>(dst + 8 * d) = make_float2(o[d][2 * h], o[d][2 * h + 1]);
            }
        }
    } while (walk.next() && walk.inside());
}

template <int D>
cudaError_t launch_d(const AttendLaunch &L, cudaStream_t stream)
{
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess)
        return e;
    const size_t smem = sizeof(SmemF32<D>);
    if (cached_occupancy(reinterpret_cast<void *>(attend_f32_kernel<D>), device, smem, smem, kF32Threads) <= 0)
        return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)L.ctas);
    cfg.blockDim = dim3(kF32Threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attend_f32_kernel<D>, L.p);
    return e;
}

// ---- the merge of cut items --------------------------------------------------------
constexpr int kMergeWarps = 8;
constexpr int kMergeRows = 16;  // rows per CTA

// CTA (c, y): rows [y kMergeRows, ..) of the item that CTA c + 1 of the attention cut first.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kMergeWarps) attend_merge_kernel(const __grid_constant__ AttendParams p)
{
    constexpr int kE = D / 32;
    dev::grid_dependency_wait();
    dev::grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cta = blockIdx.x + 1;
    const AttendCut c = p.cuts[cta];
    const int num = c.parts > 0 ? c.tokens * p.heads_per_item : 0;
    for (int r = blockIdx.y * kMergeRows + warp; r < min(num, (int)(blockIdx.y + 1) * kMergeRows); r += kMergeWarps) {
        const int tok = r / p.heads_per_item, head = r - tok * p.heads_per_item;
        if (head >= c.heads)
            continue;
        // part 0 is the second slot of the CTA before, the others the first slots from `cta` on
        auto row_of = [&](int part) {
            return part == 0 ? attend_part_row(p, cta - 1, 1) + r : attend_part_row(p, cta + part - 1, 0) + r;
        };
        // Two passes: the maximum over the parts, then 32 parts at a time, their weights a lane each.
        // (A row's parts follow one another, so 8 loads are put in flight at once.)
        float m = -INFINITY;
        for (int i = lane; i < c.parts; i += 32)
            m = fmaxf(m, p.part_ml[row_of(i)].x);
        m = dev::warp_max(m);
        const float base = m == -INFINITY ? 0.f : m;
        float l = 0.f, o[kE] = {};
        for (int i0 = 0; i0 < c.parts; i0 += 32) {
            float weight = 0.f;
            if (i0 + lane < c.parts) {
                const float2 ml = p.part_ml[row_of(i0 + lane)];
                weight = exp2f(ml.x - base);
                l += weight * ml.y;
            }
            const int n = min(c.parts - i0, 32);
#pragma unroll 8
            for (int i = 0; i < n; ++i) {
                const float w = __shfl_sync(0xffffffffu, weight, i);
                const float *src = p.part_o + row_of(i0 + i) * D + lane * kE;
                if constexpr (kE == 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(src);
                    o[0] += w * x.x;
                    o[1] += w * x.y;
                    o[2] += w * x.z;
                    o[3] += w * x.w;
                } else {
                    const float2 x = *reinterpret_cast<const float2 *>(src);
                    o[0] += w * x.x;
                    o[1] += w * x.y;
                }
            }
        }
        l = dev::warp_sum(l);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const size_t row = (size_t)(c.token0 + tok) * p.num_q_heads + c.head0 + head;
        T *dst = static_cast<T *>(p.out) + row * D + lane * kE;
        T x[kE];
#pragma unroll
        for (int e = 0; e < kE; ++e)
            x[e] = dev::from_float<T>(o[e] * inv);
        if constexpr (sizeof(x) == 16)
            *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(x);
        else if constexpr (sizeof(x) == 8)
            *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<const uint2 *>(x);
        else
            *reinterpret_cast<uint32_t *>(dst) = *reinterpret_cast<const uint32_t *>(x);
        if (p.lse && lane == 0)
            p.lse[row] = attend_lse<T>(m, l);
    }
}

template <typename T, int D>
cudaError_t launch_merge_d(const AttendLaunch &L, cudaStream_t stream)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(L.ctas - 1), (unsigned)((L.p.part_rows + kMergeRows - 1) / kMergeRows));
    cfg.blockDim = dim3(32 * kMergeWarps);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attend_merge_kernel<T, D>, L.p);
}

}  // namespace

cudaError_t launch_attend_f32(const AttendLaunch &L, cudaStream_t stream)
{
    return L.head_dim == 64 ? launch_d<64>(L, stream) : launch_d<128>(L, stream);
}
cudaError_t launch_attend_merge(const AttendLaunch &L, int dtype, cudaStream_t stream)
{
    if (L.ctas < 2)
        return cudaSuccess;
    const bool narrow = L.head_dim == 64;
    if (dtype == PA_F32)
        return narrow ? launch_merge_d<float, 64>(L, stream) : launch_merge_d<float, 128>(L, stream);
    if (dtype == PA_F16)
        return narrow ? launch_merge_d<__half, 64>(L, stream) : launch_merge_d<__half, 128>(L, stream);
    return narrow ? launch_merge_d<__nv_bfloat16, 64>(L, stream) : launch_merge_d<__nv_bfloat16, 128>(L, stream);
}

}  // namespace pagedkv
