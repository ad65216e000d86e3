// Decode attention over the 8-bit paged cache (sm_103a).
//
// The cache holds e4m3 codes and one fp32 scale per (block, kv head) for K and one
// for V (layout: pa_internal.h, q8_layout).  With ks, vs the scales of token t's
// block, the kernel computes
//     s_t = scale * ks * dot(q, K8_t),   out = sum_t exp(s_t - m) vs V8_t / sum_t exp(s_t - m)
// The schedule is pa_decode's balanced split, and the walk over the stream of
// (sequence, kv head, head group) units and the work items are its code (pa_decode.cuh);
// the producer, the scale warp, the consumers and the merges are this file's.
//
// What bounds it: the bytes of the codes, half of a 16-bit cache's; at G = 8 heads per
// kv head that is 8 multiply-adds per byte, far below the tensor pipes' rate.  Of 6682 GB/s
// (the measured copy) a batch of 2.0 GB (32 sequences, 32 / 8 heads) reaches 101%, one of
// 0.86 GB (64 ragged sequences, 64 / 8 heads) 92%, back to back.  Small batches are bound
// by their chain of latencies: 5.6 us for 50 tokens of one sequence, most of it the launch,
// lengths, table entry and first tile one after another, and 2 to 3 us more where units are
// cut, for the parts' stores, counts and merge.
//
// Conversions.  Every e4m3 value is an fp16 value, so K8 and V8 are widened to fp16
// exactly (cvt.f16x2.e4m3x2, two codes at a time) and both products run on
// mma.sync.m16n8k16 with fp16 operands and fp32 accumulators.  What is rounded:
//   q    each row is multiplied by a power of two that brings its largest element into
//        [2^10, 2^11), then rounded to fp16.  fp16 queries lose nothing (elements more
//        than 2^24 below the largest aside), bf16 ones neither (8 significant bits);
//        fp32 ones are split into two fp16 terms, 22 significant bits.
//   p vs the probability times V's scale, over a reference (Scales, below) that makes it at
//        most 2, enters as 2^14 times that: the fp16 rounding is at most 2^-11 of the value,
//        or 2^-39 of the reference.  fp32 outputs take it as two fp16 terms, 2^-22 of the
//        value or as little.  The sum of p is kept in fp32 from unrounded values.
// Scores, sums, running maxima and outputs are fp32; fp32 outputs also add each
// stage's products to the running output with an fp32 add, since the tensor pipe's own
// accumulation truncates.
//
// Scales.  ks multiplies the fp32 scores.  vs = 2^e f, 1/2 < f <= 1, multiplies p before its
// rounding, over 2^k mu.  mu is the mantissa (1 <= mu < 2) of the first vs that is not 0,
// so that scales that are alike but for powers of two round nothing.  k is the largest e
// the warp has met in the item, as long as the e lie within kSpread of each other: then
// each row's largest product is within that of the reference.  Scales that are further
// apart, or 0 beside others (the scores' maximum may be a token that adds nothing), take a
// slower path from there on, as a block whose vs is large while its p is nothing must not
// push the blocks that count out of fp16's range: each row has a second reference beside
// the scores' maximum m, w = the largest s + e, and a k of its own, ceil(w - m); the
// products are 2^(s - m + e - k) f / mu, the power taken as a whole (p alone may be below
// fp32's range although the product counts), and the accumulator follows new references by
// 2^(m - m' + k - k').  (16 sequences of 2000 tokens, 104 / 8 heads, fp16: 32.3 us, with
// scales 10 binades apart 35.3; 64 sequences, 64 / 8 heads, bf16: 140.0 and 145.1.  Rows'
// own k throughout took 35.5 of the former.)
//
// Layout of the products (16 tokens at a time).  S^T[token x row] = K Q^T: row r of the
// A tile is token 4 (r / 2) + r % 2 for r < 8 and that plus 2 for r >= 8, and the k order
// gives lane t of a row's four lanes the row's bytes [t D / 4, (t + 1) D / 4): a lane's
// share of a K row is one or two 16-byte shared loads, each word four consecutive k.
// O^T[dim x row] += V^T P^T: ldmatrix's 8-bit transposing form returns, per lane, four
// consecutive tokens of one dim; the token order above makes its low and high halves
// the A fragment's k columns that the score fragment's rows stand for, so P^T needs only
// a movmatrix transpose per 8 x 8 half, as in the 16-bit kernel.
#pragma once

#include "pa_decode.cuh"

namespace pagedkv {

#ifndef PA_Q8_STAGE_BYTES
#define PA_Q8_STAGE_BYTES 8192  // a ring stage: 32 tokens of 128 dims, 64 of 64
#endif
#ifndef PA_Q8_RING_BYTES
#define PA_Q8_RING_BYTES 81920  // shared memory of the stage ring (two CTAs per SM)
#endif

// NT: groups of 8 query rows an item may have (1 or 2).  The ring is as large as the
// residency leaves room for beside the merge rows: two CTAs per SM, or one for fp32 with
// 16 rows, whose registers allow no more.  (16 sequences of 2000 tokens, 104 / 8 heads, 128
// dims: 30.7 us on two CTAs with 64 KB each, 34.8 on one with 80 KB; fp32 with 64 / 8
// heads 23.3 and 29.4; fp32 with 104 / 8 37.1 on one CTA with 128 KB, 47.1 on two.)
template <typename T, int D, int BS, int NT>
struct Cfg8 {
    static constexpr int kCtas = sizeof(T) == 4 && NT == 2 ? 1 : 2;
    static constexpr int kRing = kCtas == 1                                    ? 131072
                                 : D == 128 && (NT == 2 || sizeof(T) == 4) ? 65536
                                                                           : PA_Q8_RING_BYTES;
    // Item descriptors in flight: one per consumer warp where a warp may have an item to
    // itself, room permitting.
    static constexpr int kSlots = NT == 1 ? 4 : kItemSlots;
    static constexpr int kTile = BS * D;          // K (or V) codes of one (block, kv head)
    static constexpr int kRecord = 2 * kTile;     // K tile, then V tile
    static constexpr int kStageTokens = PA_Q8_STAGE_BYTES / (2 * D);
    static constexpr int kBPS = kStageTokens / BS;
    static constexpr int kStageBytes = kBPS * kRecord;
    static constexpr int kStages = kRing / kStageBytes;
    // A warp gets ahead of another by kSlots items of one stage at most (they share the
    // item slots), or by one round of stages: less than a ring, which the waits rely on.
    static_assert(kStages >= kSlots + kConsumerWarps, "the warps stay within one ring of each other");
    static_assert(kStageTokens % BS == 0 && 32 % kBPS == 0, "a stage is a whole number of blocks");
    static_assert(kTile % 1024 == 0, "tiles start on the swizzle's 1024-byte period");
};

// Byte offset, in a tile as the 128-byte-swizzled copy leaves it, of 16-byte unit u of
// token `tok`'s D codes: 128-byte row tok * D / 128, units swizzled by the row's number.
template <int D>
__device__ __forceinline__ uint32_t tile_unit(int tok, int u)
{
    const int row = D == 128 ? tok : tok >> 1;
    const int unit = D == 128 ? u : ((tok & 1) * 4 + u);
    return (uint32_t)(row * 128 + ((unit ^ (row & 7)) << 4));
}

// Stream positions charged per unit for its fixed cost, in this kernel's ring stages
// (8 KB, half of pa_decode's at 128 dims).  With 4, 6, 8, 10, 12 and 16: 64 ragged sequences
// of 64 / 8 heads take 143, 140.4, 139.6, 139.4, 139.4 and 140.4 us, 8 of 40 / 40 heads 23.6,
// 23.9, 23.7, 23.7, 24.2 and 24.9, 37 of 39 / 3 heads 19.5, 18.7, 18.4, 18.1, 18.0 and 18.3.
constexpr int kUnitCost8 = 10;
// Half of them lie before the unit's stages and half behind: both parts of a unit cut in
// the middle store, count and merge.  (152 units of 26 stages on 304 CTAs, each cut once:
// 15.8 us with all of the charge before the stages, 13.8 with half.)
constexpr int kLead8 = kUnitCost8 / 2;

constexpr int kThreads8 = kThreads + 32;  // one warp more than pa_decode: the scales'

constexpr int kMergeRows = 4;  // merge rows at least: merge8 works in them

// Shared memory: as make_layout, with the scales of a stage's blocks and the range of their
// exponents (8 bytes each) in the place of the fused append's rows.
__host__ __device__ inline SmemLayout make_layout8(int stages, int stage_bytes, int bps, int slots, int rows,
                                                   int D, int elem_bytes)
{
    SmemLayout L;
    uint32_t o = (uint32_t)stages * (uint32_t)stage_bytes;
    L.acc = o;
    o += (uint32_t)(kConsumerWarps * (rows > kMergeRows ? rows : kMergeRows) * (D + kAccPad) * 4);
    L.ml = o;
    o += kConsumerWarps * kHeadsPerItem * 2 * 4;
    o = (o + 127u) & ~127u;
    L.pfx = o;
    L.items = o;
    o += (uint32_t)slots * 64u;
    L.q = o;
    o += (uint32_t)(slots * (rows <= kNarrowRows ? kNarrowRows : kHeadsPerItem) * D * elem_bytes);
    L.newrow = o;  // the scales
    o += (uint32_t)(stages * (bps + 1) * 8);
    L.newinfo = o;
    o = (o + 15u) & ~15u;
    L.bars = o;  // as make_layout's, then one per stage for its scales
    o += (3u * (uint32_t)stages + 2u * (uint32_t)slots + 1u) * 8u;
    o = (o + 15u) & ~15u;
    L.flag = o;  // as make_layout's, then a second merge flag
    o += 16u + 4u * kConsumerWarps + 4u;
    o = (o + 15u) & ~15u;
    L.blk = o;
    o += 32u * 4u;
    L.total = o + 1024u;
    return L;
}

// ---------------------------------------------------------------------------
// Producer warp: as pa_decode's, with one tiled copy per block (K and V tiles of a kv
// head are adjacent).
// ---------------------------------------------------------------------------
template <typename T, int D, int BS, int NT>
struct Producer8 {
    // G = ceil(total / divisor) <= total: none is without (a division for each part, 38 of
    // them, kept the first copy of a single sequence's one head back by 5 us)
    static constexpr bool kCountParts = false;
    static constexpr int kUnit = kUnitCost8;
    static constexpr int kLead = kLead8;
    using C = Cfg8<T, D, BS, NT>;
    const DecodeParams &p;
    const CUtensorMap *map;
    const CtaState &c;
    int lane;
    uint32_t g;  // stages issued
    uint32_t n;  // items published
    bool failed;

    __device__ Producer8(const DecodeParams &p_, const CUtensorMap *map_, const CtaState &c_, int lane_)
        : p(p_), map(map_), c(c_), lane(lane_), g(0), n(0), failed(false)
    {
        if (lane == 0)
            dev::tma_prefetch_desc(map);
    }

    __device__ bool wait_slot(uint64_t *bar, uint32_t parity)
    {
        const int r = dev::mbar_wait_abortable(dev::smem_addr(bar), parity, p.wait_ns, c.abort);
        if (r == 0)
            raise_error(p, c.abort, PA_DEVERR_TIMEOUT_EMPTY);
        return r == 1;
    }

    __device__ bool emit(const Item &it)
    {
        constexpr uint32_t kQSlotBytes = NT * 8 * D * sizeof(T);
        const uint32_t slot = n % C::kSlots;
        int ok = 1;
        if (lane == 0) {
            ok = wait_slot(&c.item_empty[slot], ((n / C::kSlots) & 1u) ^ 1u);
            if (ok) {
                c.items[slot] = it;
                const uint32_t bytes = (uint32_t)it.rows * D * sizeof(T);
                const uint32_t fb = dev::smem_addr(&c.item_full[slot]);
                dev::mbar_arrive_expect_tx(fb, bytes);
                dev::bulk_load(dev::smem_addr(c.qslots + slot * kQSlotBytes),
                               reinterpret_cast<const T *>(p.q) +
                                   ((size_t)it.seq * p.num_q_heads + it.qrow0) * D,
                               bytes, fb);
            }
        }
        if (!__shfl_sync(0xffffffffu, ok, 0)) {
            failed = true;
            return false;
        }
        ++n;
        const int32_t *row = p.block_tables + (size_t)it.tseq * p.max_blocks;
        // one coalesced read per 32 blocks, a window ahead
        int next = it.j0 + lane < it.j1 ? row[it.j0 + lane] : -1;
        for (int jb = it.j0; jb < it.j1; jb += 32) {
            c.blk[lane] = next;
            next = jb + 32 + lane < it.j1 ? row[jb + 32 + lane] : -1;
            __syncwarp();
            uint32_t issued = 0;
            ok = 1;
            if (lane == 0)
                ok = fill_window(it, min(32, it.j1 - jb), issued);
            g += __shfl_sync(0xffffffffu, issued, 0);
            if (!__shfl_sync(0xffffffffu, ok, 0)) {
                failed = true;
                return false;
            }
        }
        return true;
    }

    // Lane 0: the stages of one window of cnt blocks (ids in c.blk).
    __device__ int fill_window(const Item &it, int cnt, uint32_t &issued)
    {
        uint32_t gg = g;
        for (int i = 0; i < cnt; i += C::kBPS, ++gg) {
            const int nbs = min(C::kBPS, cnt - i);  // blocks in this stage
            const uint32_t st = gg % C::kStages;
            if (!wait_slot(&c.empty[st], ((gg / C::kStages) & 1u) ^ 1u)) {
                issued = gg - g;
                return 0;
            }
            const uint32_t fb = dev::smem_addr(&c.full[st]);
            dev::mbar_arrive_expect_tx(fb, (uint32_t)nbs * C::kRecord);
            const uint32_t dst = dev::smem_addr(c.ring + (size_t)st * C::kStageBytes);
#pragma unroll
            for (int b = 0; b < C::kBPS; ++b) {
                if (b < nbs) {
                    const int id = c.blk[i + b];
                    // an entry outside the pool reads zeros
                    dev::tma_load_4d(dst + (uint32_t)b * C::kRecord, map, 0, 0, it.kvh,
                                     id >= 0 && id < p.num_blocks ? id : -1, fb);
                }
            }
        }
        issued = gg - g;
        return 1;
    }

    // End of the walk: as Producer::finish (every copy in flight lands before the warp
    // exits, each wait with the full bound).
    __device__ void finish()
    {
        if (lane != 0)
            return;
        for (uint32_t k = n > C::kSlots ? n - C::kSlots : 0; k < n; ++k)
            dev::mbar_wait(dev::smem_addr(&c.item_full[k % C::kSlots]), (k / C::kSlots) & 1u,
                           kWaitTimeoutNs);
        if (!failed) {
            const uint32_t slot = n % C::kSlots;
            if (wait_slot(&c.item_empty[slot], ((n / C::kSlots) & 1u) ^ 1u)) {
                c.items[slot].seq = -1;
                dev::mbar_arrive(dev::smem_addr(&c.item_full[slot]));
            } else {
                failed = true;
            }
        }
        for (uint32_t q = g > C::kStages ? g - C::kStages : 0; q < g; ++q)
            dev::mbar_wait(dev::smem_addr(&c.full[q % C::kStages]), (q / C::kStages) & 1u, kWaitTimeoutNs);
    }
};

// 2^n, for n of -149 .. 127.
__device__ __forceinline__ float pow2(int n)
{
    return __uint_as_float(n >= -126 ? (uint32_t)(n + 127) << 23 : 1u << (n + 149));
}

// e of a scale 2^e f with 1/2 < f <= 1, as a float: -inf for 0, at least -126 otherwise.
__device__ __forceinline__ float scale_exponent(float x)
{
    return x == 0.f ? -INFINITY : (float)((int)((__float_as_uint(x) + 0x7fffffu) >> 23) - 127);
}

// ---------------------------------------------------------------------------
// Scale warp: walks the same items as the producer and brings each stage's scales into
// shared memory by plain loads.  (A 16-byte bulk copy of them behind every block's tiles
// made the producer the bottleneck: 189 us instead of 161 for 64 sequences of 64 / 8
// heads, 16-token blocks, with the copy merely left out.)  A lane has one block of a
// window of 32: the loads of the next window's ids and scales are in flight while the
// stages of this one are handed over.
// ---------------------------------------------------------------------------
template <typename T, int D, int BS, int NT>
struct ScaleWarp {
    static constexpr bool kCountParts = false;
    static constexpr int kUnit = kUnitCost8;
    static constexpr int kLead = kLead8;
    using C = Cfg8<T, D, BS, NT>;
    const DecodeParams &p;
    const Q8Params &q8;
    const CtaState &c;
    uint64_t *sfull;  // per stage: its scales are in shared memory
    int lane;
    uint32_t g;  // stages handed over

    __device__ ScaleWarp(const DecodeParams &p_, const Q8Params &q8_, const CtaState &c_, uint64_t *sfull_,
                         int lane_)
        : p(p_), q8(q8_), c(c_), sfull(sfull_), lane(lane_), g(0)
    {
    }

    __device__ int block_id(const Item &it, const int32_t *row, int j) const
    {
        return j < it.j1 ? row[j] : -1;
    }
    __device__ float2 scales_of(const Item &it, int id) const
    {
        if (id < 0 || id >= p.num_blocks)
            return make_float2(0.f, 0.f);  // reads zeros, as the producer's copy does
        return __ldcg(reinterpret_cast<const float2 *>(q8.scales + (size_t)id * q8.block_bytes) + it.kvh);
    }

    // Largest and smallest e of the V scales (scale_exponent; a block past the item is
    // neither) of the lane's stage, whose blocks are kBPS consecutive lanes'.
    static __device__ float2 range_of(float vs, bool past)
    {
        float2 e = make_float2(scale_exponent(vs), past ? INFINITY : scale_exponent(vs));
#pragma unroll
        for (int o = 1; o < C::kBPS; o <<= 1) {
            e.x = fmaxf(e.x, __shfl_xor_sync(0xffffffffu, e.x, o));
            e.y = fminf(e.y, __shfl_xor_sync(0xffffffffu, e.y, o));
        }
        return e;
    }

    __device__ bool emit(const Item &it)
    {
        const int32_t *row = p.block_tables + (size_t)it.tseq * p.max_blocks;
        int id = block_id(it, row, it.j0 + lane);
        int next_id = block_id(it, row, it.j0 + 32 + lane);
        float2 s = scales_of(it, id);
        // A split unit's counter takes this launch's epoch here, so that the parts' counts
        // need no exchange (0.4 us of 12 where two parts of every unit end together): a value
        // read as another epoch's changes to this one's only.
        unsigned long long *const ctr = p.counters + it.c_first;
        if (it.partial && lane == 0) {
            const unsigned long long seen = *reinterpret_cast<volatile unsigned long long *>(ctr);
            if ((unsigned int)(seen >> 32) != p.epoch)
                atomicCAS(ctr, seen, (unsigned long long)p.epoch << 32);
        }
        for (int jb = it.j0; jb < it.j1; jb += 32) {
            const float2 next_s = scales_of(it, next_id);
            next_id = block_id(it, row, jb + 64 + lane);
            const int cnt = min(32, it.j1 - jb);
            const float2 range = range_of(s.y, lane >= cnt);
            for (int i = 0; i < cnt; i += C::kBPS, ++g) {
                const uint32_t st = g % C::kStages;
                int ok = 1;
                if (lane == 0)
                    ok = dev::mbar_wait_abortable(dev::smem_addr(&c.empty[st]), ((g / C::kStages) & 1u) ^ 1u,
                                                  p.wait_ns, c.abort);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (ok != 1) {
                    if (ok == 0 && lane == 0)
                        raise_error(p, c.abort, PA_DEVERR_TIMEOUT_EMPTY);
                    return false;
                }
                // (blocks past the item: zeros)
                float2 *const dst = reinterpret_cast<float2 *>(c.newrow) + st * (C::kBPS + 1);
                if (lane >= i && lane < i + C::kBPS)
                    dst[lane - i] = s;
                if (lane == i)
                    dst[C::kBPS] = range;
                __syncwarp();
                if (lane == 0)
                    dev::mbar_arrive(dev::smem_addr(&sfull[st]));
            }
            s = next_s;
        }
        return true;
    }
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// N consecutive elements, 16 bytes at a time, as fp32.
template <typename T, int N>
__device__ __forceinline__ void load_row(float (&x)[N], const T *src)
{
    constexpr int E = 16 / (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < N / E; ++i) {
        const uint4 w = reinterpret_cast<const uint4 *>(src)[i];
        const T *e = reinterpret_cast<const T *>(&w);
#pragma unroll
        for (int k = 0; k < E; ++k)
            x[i * E + k] = to_float(e[k]);
    }
}

// k of a row whose references are m and w: at least -126, where p vs is below fp32's
// normal range altogether (also without any w); at most 128, as w <= m + 128.
__device__ __forceinline__ float shift_of(float w, float m) { return fmaxf(ceilf(w - m), -126.f); }

// Four consecutive outputs in the storage type.
template <typename T>
__device__ __forceinline__ void store4(T *dst, const float (&x)[4])
{
    if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float4 *>(dst) = make_float4(x[0], x[1], x[2], x[3]);
    else
        *reinterpret_cast<uint2 *>(dst) = make_uint2(dev::Mma<T>::pack(x[0], x[1]), dev::Mma<T>::pack(x[2], x[3]));
}

// Hand an item slot back, once every read of it has completed: `all` is made of what the
// warp's lanes read of the query rows.
__device__ __forceinline__ void release_item(const CtaState &c, const Item &it, uint32_t slot, int warp, int lane,
                                             uint32_t all)
{
    all ^= (uint32_t)(it.seq ^ it.kvh ^ it.hg ^ it.len ^ it.j0 ^ it.j1 ^ it.qrow0 ^ it.rows ^ it.partial ^
                      it.prow0 ^ it.tseq ^ it.packed ^ it.c_first ^ it.nparts) ^
           it.total_lo ^ it.total_hi;
    all = __reduce_xor_sync(0xffffffffu, all);
    if (lane == 0)
        dev::settle_loads(&c.sink[warp], all);
    __syncwarp();
    if (lane == 0)
        dev::mbar_arrive(dev::smem_addr(&c.item_empty[slot]));
}

// Byte offset of token tile mt (16 tokens) in a stage's K codes (V's lie kTile behind): a
// multiple of 1024, so that the swizzle of a lane's share does not depend on mt.
template <int D, int BS>
__device__ __forceinline__ constexpr uint32_t tile_offset(int mt)
{
    return (uint32_t)((mt * 16 / BS) * 2 * BS * D + (mt * 16 % BS) * D);
}

// ---------------------------------------------------------------------------
// One item on one consumer warp (its share of the item's stages).  NT: 8-row groups of
// query rows.  Ends with the warp's partial rows in its merge area or, `alone`, with the
// item's output.  `seen`: the counter of a split unit, read by thread 0 on the way.
// ---------------------------------------------------------------------------
template <typename T, int D, int BS, int NT>
__device__ __forceinline__ bool consume_item8(const DecodeParams &p, const CtaState &c, const Item &it,
                                              uint64_t *sfull, uint32_t slot, uint32_t &g, int warp, int lane,
                                              int rows_cap, bool alone, unsigned long long &seen)
{
    using C = Cfg8<T, D, BS, NT>;
    constexpr bool kSplit = sizeof(T) == 4;  // two fp16 terms for q and p
    constexpr int QT = kSplit ? 2 : 1;
    constexpr int TS = C::kStageTokens;
    constexpr int MT = TS / 16;   // 16-token tiles of a stage
    constexpr int KS = D / 16;    // k-steps of K Q^T = words of a lane's share of a K row
    constexpr int DM = D / 16;    // 16-dim tiles of O^T
    constexpr int SA = D + kAccPad;
    constexpr uint32_t kQSlotBytes = NT * 8 * D * sizeof(T);
    constexpr int kUp = 14;         // products are held times 2^kUp
    constexpr float kSpread = 6.f;  // binades over which all e lie, or rows take a k each
    const int q4 = lane & 3;       // fragment columns: query rows 8 nt + 2 q4, + 1
    const int r8 = lane >> 2;      // fragment row
    const int tok0 = 4 * (r8 >> 1) + (r8 & 1);  // this lane's tokens of a tile: tok0, tok0 + 2
    // Its shares of them in a K tile (a row's next 16-byte unit is the address ^ 16), and its
    // row of a V tile's first 32 dims (the next 32: ^ 32).  Tiles start on multiples of
    // 1024 bytes, so the exclusive or acts on the swizzled unit alone.
    const uint32_t koff0 = tile_unit<D>(tok0, q4 * (D / 64)), koff1 = tile_unit<D>(tok0 + 2, q4 * (D / 64));
    const uint32_t voff = tile_unit<D>(lane & 15, lane >> 4);
    const uint32_t ring = dev::smem_addr(c.ring), scales = dev::smem_addr(c.newrow);

    // Q^T as the B operand, and the factor each row's scores take
    uint32_t qb[NT][QT][KS][2];
    float fa[NT], fb[NT];
    {
        uint32_t all = 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float x[D / 4];
            const T *src = reinterpret_cast<const T *>(c.qslots + slot * kQSlotBytes) +
                           (size_t)(nt * 8 + r8) * D + q4 * (D / 4);
            load_row<T, D / 4>(x, src);
            const bool live = nt * 8 + r8 < it.rows;
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < D / 4; ++i) {
                x[i] = live ? x[i] : 0.f;
                top = fmaxf(top, fabsf(x[i]));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^(10 - floor(log2 top)) and its inverse, by exponent bits
            const int e = min(max((int)(__float_as_uint(top) >> 23), 11), 254);
            const float up = __uint_as_float((uint32_t)(264 - e) << 23);
            const float down = top == 0.f ? 1.f : __uint_as_float((uint32_t)(e - 10) << 23);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float y0 = x[4 * ks + 2 * h] * up, y1 = x[4 * ks + 2 * h + 1] * up;
                    const uint32_t hi = dev::Mma<__half>::pack(y0, y1);
                    qb[nt][0][ks][h] = hi;
                    all ^= hi;
                    if constexpr (kSplit) {
                        const __half2 hh = *reinterpret_cast<const __half2 *>(&hi);
                        qb[nt][1][ks][h] =
                            dev::Mma<__half>::pack(y0 - __low2float(hh), y1 - __high2float(hh));
                    }
                }
            }
            fa[nt] = __shfl_sync(0xffffffffu, down, 8 * q4) * p.scale_log2;
            fb[nt] = __shfl_sync(0xffffffffu, down, 8 * q4 + 4) * p.scale_log2;
        }
        release_item(c, it, slot, warp, lane, all);
    }

    float o[NT][DM][4];
    float ma[NT], mb[NT], la[NT], lb[NT];  // reference and sum of rows 2 q4, 2 q4 + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        ma[nt] = mb[nt] = -INFINITY;
        la[nt] = lb[nt] = 0.f;
#pragma unroll
        for (int i = 0; i < DM; ++i)
            o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    }
    float mu = 0.f;                              // mantissa of the first vs that is not 0
    float e_top = -INFINITY, e_low = INFINITY;   // largest and smallest e so far
    float vinv = 0.f;                            // 2^-k / mu, or 1 / mu where rows have a k each
    bool spread = false;                         // they have
    // w and k of the rows then: at the start of the warp's own merge rows (16 floats a group
    // of 8 rows; a merge row has 72 at least)
    float2 *const wk = reinterpret_cast<float2 *>(c.macc + warp * rows_cap * SA) + 2 * q4;
    const int rot = it.rot();
    const int stages = (it.j1 - it.j0 + C::kBPS - 1) / C::kBPS;
    int i = (warp - rot) & (kConsumerWarps - 1);
    if (i >= stages && threadIdx.x == 0 && it.partial)
        seen = *reinterpret_cast<volatile unsigned long long *>(p.counters + it.c_first);
    for (; i < stages; i += kConsumerWarps) {
        // the counter is read behind the warp's last stage, and looked at after it
        if (i + kConsumerWarps >= stages && threadIdx.x == 0 && it.partial)
            seen = *reinterpret_cast<volatile unsigned long long *>(p.counters + it.c_first);
        const int j = it.j0 + i * C::kBPS;
        const uint32_t st = (g + i) % C::kStages, phase = ((g + i) / C::kStages) & 1u;
        // The scales' barrier first.  Consecutive uses of a stage may belong to different
        // warps (the ring need not be a multiple of four stages), and a wait by parity
        // must not begin while the use before is still under way: it would take the use
        // before that one for its own.  Stages' data may land out of order, so the data's
        // barrier alone would allow it.  The scale warp hands the stages over in order, each
        // after its previous use was released, so behind its barrier the data's is in the
        // right phase; and its own barrier is, because this warp has passed an earlier stage
        // or an item's end less than a ring ago.
        if (!warp_wait(p, c, &sfull[st], phase) || !warp_wait(p, c, &c.full[st], phase))
            return false;
        const int nbs = min(C::kBPS, it.j1 - j);  // blocks in this stage
        const int valid = min(nbs * BS, it.len - j * BS);
        const bool partial = valid < TS;
        const uint32_t stage = ring + st * C::kStageBytes;
        float kscale[C::kBPS], vscale[C::kBPS];  // (blocks past the item: 0)
        const uint32_t sc = scales + st * (C::kBPS + 1) * 8;
#pragma unroll
        for (int b = 0; b < C::kBPS; ++b) {
            const float2 s2 = dev::lds_f2(sc + b * 8);
            kscale[b] = s2.x;
            vscale[b] = s2.y;
        }
        const float2 range = dev::lds_f2(sc + C::kBPS * 8);
        const float top = fmaxf(e_top, range.x);
        e_low = fminf(e_low, range.y);

        // S^T = K Q^T, even and odd k-steps in accumulators of their own (shorter chains)
        float s[MT][NT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const uint32_t kt = stage + tile_offset<D, BS>(mt);
            uint32_t w0[KS], w1[KS];
#pragma unroll
            for (int u = 0; u < D / 64; ++u) {
                dev::lds128(&w0[4 * u], (kt + koff0) ^ (uint32_t)(u << 4));
                dev::lds128(&w1[4 * u], (kt + koff1) ^ (uint32_t)(u << 4));
            }
            float s2[NT][2][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s2[nt][0][e] = s2[nt][1][e] = 0.f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t a[4];
                dev::e4m3x4_to_f16x4(w0[ks], a[0], a[2]);
                dev::e4m3x4_to_f16x4(w1[ks], a[1], a[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int t = 0; t < QT; ++t)
                        dev::Mma<__half>::run(s2[nt][ks & 1], a, qb[nt][t][ks][0], qb[nt][t][ks][1]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[mt][nt][e] = s2[nt][0][e] + s2[nt][1][e];
        }

        // Scale and mask.  A lane compares its own scores with the reference: only where
        // one passes it by more than 1 do the lanes look for the maximum, and the warp
        // takes a new reference.
        bool raise = top > e_top;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const float ksc = kscale[mt * 16 / BS];
                const float ga = fa[nt] * ksc, gb = fb[nt] * ksc;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float &xa = s[mt][nt][2 * h], &xb = s[mt][nt][2 * h + 1];
                    xa *= ga;
                    xb *= gb;
                    if (partial && mt * 16 + tok0 + 2 * h >= valid)
                        xa = xb = -INFINITY;
                    raise |= xa > ma[nt] + 1.f || xb > mb[nt] + 1.f;
                }
            }
        }
        // (rows of maxima: a lane's own tokens, then the lanes of the same rows)
        auto row_max = [](float x) {
#pragma unroll
            for (int o_ = 4; o_ < 32; o_ <<= 1)
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o_));
            return x;
        };
        auto rescale = [&](int nt, float ca, float cb) {
#pragma unroll
            for (int i = 0; i < DM; ++i) {
                o[nt][i][0] *= ca;
                o[nt][i][1] *= cb;
                o[nt][i][2] *= ca;
                o[nt][i][3] *= cb;
            }
        };
        float counted = 1.f;
        auto find_mu = [&] {
#pragma unroll
            for (int b = 0; b < C::kBPS; ++b)
                if (mu == 0.f && vscale[b] > 0.f)
                    mu = vscale[b] < FLT_MIN
                             ? 1.f
                             : __uint_as_float((__float_as_uint(vscale[b]) & 0x7fffffu) | 0x3f800000u);
        };
        if (__builtin_expect(top - e_low > kSpread, 0)) {
            if (!spread) {  // from here on: what the rows hold so far is within 2^m 2^e_top
                spread = true;
                find_mu();
                vinv = 1.f / mu;
                if (r8 == 0) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        wk[nt * 8] = make_float2(ma[nt] + e_top, fmaxf(e_top, -126.f));
                        wk[nt * 8 + 1] = make_float2(mb[nt] + e_top, fmaxf(e_top, -126.f));
                    }
                }
                __syncwarp();
            }
            float vexp[C::kBPS];
#pragma unroll
            for (int b = 0; b < C::kBPS; ++b)
                vexp[b] = scale_exponent(vscale[b]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float2 old_a = wk[nt * 8], old_b = wk[nt * 8 + 1];
                float na = ma[nt], nb = mb[nt], va = old_a.x, vb = old_b.x;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const float xa = fmaxf(s[mt][nt][0], s[mt][nt][2]), xb = fmaxf(s[mt][nt][1], s[mt][nt][3]);
                    na = fmaxf(na, xa);
                    nb = fmaxf(nb, xb);
                    va = fmaxf(va, xa + vexp[mt * 16 / BS]);
                    vb = fmaxf(vb, xb + vexp[mt * 16 / BS]);
                }
                na = row_max(na);
                nb = row_max(nb);
                va = row_max(va);
                vb = row_max(vb);
                const float ka = shift_of(va, na), kb = shift_of(vb, nb);
                // (one power for both: it is at most about 2, its factors may not be finite)
                const bool fresh_a = ma[nt] == -INFINITY, fresh_b = mb[nt] == -INFINITY;
                const float da = ma[nt] - na, db = mb[nt] - nb;
                rescale(nt, fresh_a ? 0.f : exp2f(da + (old_a.y - ka)),
                        fresh_b ? 0.f : exp2f(db + (old_b.y - kb)));
                la[nt] *= fresh_a ? 0.f : exp2f(da);
                lb[nt] *= fresh_b ? 0.f : exp2f(db);
                ma[nt] = na;
                mb[nt] = nb;
                __syncwarp();
                if (r8 == 0) {
                    wk[nt * 8] = make_float2(va, ka);
                    wk[nt * 8 + 1] = make_float2(vb, kb);
                }
                // p is counted here, and the scores move by e - k for the products
                na = na == -INFINITY ? 0.f : na;
                nb = nb == -INFINITY ? 0.f : nb;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float &xa = s[mt][nt][2 * h], &xb = s[mt][nt][2 * h + 1];
                        la[nt] += dev::ex2(xa - na);
                        lb[nt] += dev::ex2(xb - nb);
                        xa += vexp[mt * 16 / BS] - ka;
                        xb += vexp[mt * 16 / BS] - kb;
                    }
            }
            e_top = top;  // (the difference never shrinks)
            counted = 0.f;
#pragma unroll
            for (int b = 0; b < C::kBPS; ++b)  // f
                vscale[b] = vscale[b] == 0.f ? 0.f : vscale[b] * pow2(-(int)vexp[b]);
        } else if (__any_sync(0xffffffffu, raise)) {
            // (e_top grows by kSpread at most, or from -inf, when there is nothing yet)
            const float cv = e_top == top || e_top == -INFINITY ? 1.f : pow2((int)(e_top - top));
            find_mu();
            vinv = mu == 0.f ? 0.f : pow2(-(int)top) / mu;
            e_top = top;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float na = ma[nt], nb = mb[nt];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    na = fmaxf(na, fmaxf(s[mt][nt][0], s[mt][nt][2]));
                    nb = fmaxf(nb, fmaxf(s[mt][nt][1], s[mt][nt][3]));
                }
                na = row_max(na);
                nb = row_max(nb);
                // (no finite score yet: nothing to rescale)
                const float ca = ma[nt] == -INFINITY ? 0.f : exp2f(ma[nt] - na);
                const float cb = mb[nt] == -INFINITY ? 0.f : exp2f(mb[nt] - nb);
                ma[nt] = na;
                mb[nt] = nb;
                la[nt] *= ca;
                lb[nt] *= cb;
                rescale(nt, ca * cv, cb * cv);
            }
        }

        // P^T as the B operand: 2^kUp p vs 2^-k / mu, rounded, transposed
        uint32_t pb[MT][NT][QT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float na = ma[nt] == -INFINITY ? 0.f : ma[nt], nb = mb[nt] == -INFINITY ? 0.f : mb[nt];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const float vs = vscale[mt * 16 / BS] * vinv * (float)(1 << kUp);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float ea = dev::ex2(s[mt][nt][2 * h] - na), eb = dev::ex2(s[mt][nt][2 * h + 1] - nb);
                    la[nt] = fmaf(ea, counted, la[nt]);
                    lb[nt] = fmaf(eb, counted, lb[nt]);
                    const float ya = ea * vs, yb = eb * vs;
                    const uint32_t hi = dev::Mma<__half>::pack(ya, yb);
                    pb[mt][nt][0][h] = dev::movmatrix_trans(hi);
                    if constexpr (kSplit) {
                        const __half2 hh = *reinterpret_cast<const __half2 *>(&hi);
                        pb[mt][nt][1][h] = dev::movmatrix_trans(
                            dev::Mma<__half>::pack(ya - __low2float(hh), yb - __high2float(hh)));
                    }
                }
            }
        }

        // O^T += V^T P^T, 32 dims (two 16 x 16 matrices of codes) at a time
#pragma unroll
        for (int dp = 0; dp < DM / 2; ++dp) {
            float loc[NT][2][4];
            if constexpr (kSplit) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        loc[nt][0][e] = loc[nt][1][e] = 0.f;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                uint32_t v[4];
                dev::ldsm_b8_x2_trans((stage + C::kTile + tile_offset<D, BS>(mt) + voff) ^ (uint32_t)(dp << 5), v[0],
                                      v[1], v[2], v[3]);
                if (partial) {
                    // rows past the context may hold anything (NaN): zero their codes
                    const int left = min(max(valid - mt * 16 - 4 * q4, 0), 4);
                    const uint32_t keep = left == 4 ? 0xffffffffu : (1u << (8 * left)) - 1u;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] &= keep;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t a[4];
                    dev::e4m3x4_to_f16x4(v[2 * h], a[0], a[2]);
                    dev::e4m3x4_to_f16x4(v[2 * h + 1], a[1], a[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int t = 0; t < QT; ++t) {
                            if constexpr (kSplit)
                                dev::Mma<__half>::run(loc[nt][h], a, pb[mt][nt][t][0], pb[mt][nt][t][1]);
                            else
                                dev::Mma<__half>::run(o[nt][2 * dp + h], a, pb[mt][nt][t][0], pb[mt][nt][t][1]);
                        }
                }
            }
            if constexpr (kSplit) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[nt][2 * dp + h][e] += loc[nt][h][e];
            }
        }
        __syncwarp();
        if (lane == 0)
            dev::mbar_arrive(dev::smem_addr(&c.empty[st]));
    }

    g += stages;

    // Partial rows of this warp: back from 2^kUp p vs 2^-k / mu in two steps (2^(k - kUp) alone
    // is exact also where it is below the normal range).
    float *mine = c.macc + warp * rows_cap * SA;
    float ua[NT], ub[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        ua[nt] = ub[nt] = pow2((int)fmaxf(e_top, -126.f) - kUp);
    if (spread) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            ua[nt] = pow2((int)wk[nt * 8].y - kUp);
            ub[nt] = pow2((int)wk[nt * 8 + 1].y - kUp);
        }
        __syncwarp();  // the rows take their place
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float sa = la[nt], sb = lb[nt];
#pragma unroll
        for (int o_ = 4; o_ < 32; o_ <<= 1) {
            sa += __shfl_xor_sync(0xffffffffu, sa, o_);
            sb += __shfl_xor_sync(0xffffffffu, sb, o_);
        }
        const int ra = nt * 8 + 2 * q4, rb = ra + 1;
        if (ra < it.rows) {
#pragma unroll
            for (int dm = 0; dm < DM; ++dm) {
                mine[ra * SA + dm * 16 + r8] = o[nt][dm][0] * mu * ua[nt];
                mine[ra * SA + dm * 16 + r8 + 8] = o[nt][dm][2] * mu * ua[nt];
            }
        }
        if (rb < it.rows) {
#pragma unroll
            for (int dm = 0; dm < DM; ++dm) {
                mine[rb * SA + dm * 16 + r8] = o[nt][dm][1] * mu * ub[nt];
                mine[rb * SA + dm * 16 + r8 + 8] = o[nt][dm][3] * mu * ub[nt];
            }
        }
        if (NT == 1 && alone) {
            // the rows' sums, behind the rows
            if (r8 == 0 && ra < it.rows)
                mine[ra * SA + D] = sa;
            if (r8 == 0 && rb < it.rows)
                mine[rb * SA + D] = sb;
        } else if (r8 == 0) {
            // a NaN score makes the sum and every output NaN; the merge takes such a
            // row with a sum of 1, so that the NaN outputs, not the sum, carry it on
            const bool na = sa != sa, nb = sb != sb;
            c.mml[(warp * kHeadsPerItem + ra) * 2] =
                ra < it.rows && (na || sa > 0.f) ? (na ? 0.f : ma[nt]) : -INFINITY;
            c.mml[(warp * kHeadsPerItem + ra) * 2 + 1] = na ? 1.f : sa;
            c.mml[(warp * kHeadsPerItem + rb) * 2] =
                rb < it.rows && (nb || sb > 0.f) ? (nb ? 0.f : mb[nt]) : -INFINITY;
            c.mml[(warp * kHeadsPerItem + rb) * 2 + 1] = nb ? 1.f : sb;
        }
    }
    if (NT == 1 && alone) {
        __syncwarp();
        constexpr int LR = D / 4;  // lanes on a row
        for (int r = lane / LR; r < it.rows; r += 32 / LR) {
            const int col = lane % LR * 4;
            const float4 v = *reinterpret_cast<const float4 *>(&mine[r * SA + col]);
            const float L = mine[r * SA + D];
            float y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                y[e] = L == 0.f ? 0.f : y[e] / L;
            store4(reinterpret_cast<T *>(p.out) + ((size_t)it.seq * p.num_q_heads + it.qrow0 + r) * D + col, y);
        }
        __syncwarp();  // read before the next item's take their place
    }
    return true;
}

// The square root of a merge's weight 2^x.  Rows are multiplied by it twice: with V scales
// far apart a weight may be below fp32's range although its row counts.
__device__ __forceinline__ float root_weight(float x) { return exp2f(0.5f * x); }

// One part of a split unit joins its row's merge: M the largest log2-sum-exp of the parts
// at hand (a part without any weight, -inf, adds nothing).  A unit cut once is merged by
// finalize8 or by merge_few, as its parts happen to end; both add them in slot order with
// these operations, so that the result has the same bits either way.
__device__ __forceinline__ void add_part(float (&o)[4], float &W, float M, float lse, const float4 &v)
{
    if (lse != -INFINITY) {
        const float h = root_weight(lse - M);
        W = __fmaf_rn(h, h, W);
        o[0] = __fmaf_rn(h, __fmul_rn(h, v.x), o[0]);
        o[1] = __fmaf_rn(h, __fmul_rn(h, v.y), o[1]);
        o[2] = __fmaf_rn(h, __fmul_rn(h, v.z), o[2]);
        o[3] = __fmaf_rn(h, __fmul_rn(h, v.w), o[3]);
    }
}

// ---------------------------------------------------------------------------
// Merge the four consumer states of one item and store it, as finalize_item does, four
// columns per thread and D / 4 threads per row, so that a row's weights are computed
// once per thread.  `other` >= 0: the item completes a unit cut once; the other part's
// rows lie there, and the merged rows go to the output at once.
// ---------------------------------------------------------------------------
template <typename T, int D>
__device__ __forceinline__ void finalize8(const DecodeParams &p, const Item &it, const float *acc, const float *ml,
                                          int rows_cap, int tid, int other)
{
    constexpr int S = D + kAccPad;
    constexpr int LR = D / 4;  // threads on a row: a warp or half of one
    for (int r = tid / LR; r < it.rows; r += 32 * kConsumerWarps / LR) {
        const int col = tid % LR * 4;
        float lse2 = -INFINITY;
        float4 o2 = make_float4(0.f, 0.f, 0.f, 0.f);
        if (other >= 0) {
            lse2 = __ldcg(p.part_lse + other + r);
            o2 = __ldcg(reinterpret_cast<const float4 *>(p.part_o + (size_t)(other + r) * D + col));
        }
        float mc[kConsumerWarps], lc[kConsumerWarps];
        float4 v[kConsumerWarps];
        float M = -INFINITY;
#pragma unroll
        for (int c = 0; c < kConsumerWarps; ++c) {
            const float2 x = *reinterpret_cast<const float2 *>(&ml[(c * kHeadsPerItem + r) * 2]);
            mc[c] = x.x;
            lc[c] = x.y;
            v[c] = *reinterpret_cast<const float4 *>(&acc[(c * rows_cap + r) * S + col]);
            M = fmaxf(M, mc[c]);
        }
        float L = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < kConsumerWarps; ++c) {
            if (mc[c] != -INFINITY) {  // (a warp without stages left no rows)
                const float h = root_weight(mc[c] - M);
                L += h * h * lc[c];
                o[0] += h * (h * v[c].x);
                o[1] += h * (h * v[c].y);
                o[2] += h * (h * v[c].z);
                o[3] += h * (h * v[c].w);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = L > 0.f ? o[e] / L : 0.f;
        const float lse = L > 0.f ? M + log2f(L) : -INFINITY;
        if (it.partial && other < 0) {
            const size_t pr = (size_t)it.prow0 + r;
            *reinterpret_cast<float4 *>(p.part_o + pr * D + col) = make_float4(o[0], o[1], o[2], o[3]);
            if (col == 0)
                p.part_lse[pr] = lse;
            continue;
        }
        if (other >= 0) {  // both parts by slot, not by which of them ended first
            const bool ahead = it.prow0 < other;
            const float M2 = fmaxf(lse, lse2);
            float W = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
            const float4 mine = make_float4(o[0], o[1], o[2], o[3]);
            add_part(y, W, M2, ahead ? lse : lse2, ahead ? mine : o2);
            add_part(y, W, M2, ahead ? lse2 : lse, ahead ? o2 : mine);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = W > 0.f ? y[e] / W : 0.f;
        }
        store4(reinterpret_cast<T *>(p.out) + ((size_t)it.seq * p.num_q_heads + it.qrow0 + r) * D + col, o);
    }
}

constexpr int kFlight = 8;  // parts of a split unit that a thread reads at once

// Floats of the merge rows (make_layout8) that merge8 may use.
__device__ __forceinline__ int merge_room(int rows_cap, int D)
{
    return kConsumerWarps * max(rows_cap, kMergeRows) * (D + kAccPad);
}

// Merge the partials of a split unit into its output rows by the log-sum-exp rule, all
// consumer warps together, where they are many: every (row, part)'s log2-sum-exp in one
// round of loads, a row's weights by one warp, then the weighted rows, D / 4 threads per row
// with two rows and eight parts of each in flight; with fewer rows than such groups of
// threads, several groups share a row's parts.  `room`: the merge rows, free by now.  False on a timeout.
template <typename T, int D>
__device__ __forceinline__ bool merge8(const DecodeParams &p, const Item &it, const CtaState &c, uint32_t &sph,
                                       int warp, int lane, float *room)
{
    constexpr int LR = D / 4;                             // threads on a row
    constexpr int kGroups = 32 * kConsumerWarps / LR;
    const int n = it.nparts, tid = warp * 32 + lane;
    // every CTA up to G has positions, so the parts' slots are consecutive (split_slot)
    auto slot = [&](int i) { return (2 * (it.c_first + i) + (i == 0 ? 1 : 0)) * kHeadsPerItem; };
    for (int k = tid; k < it.rows * n; k += 4 * 32 * kConsumerWarps) {
        float lse[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int x = min(k + u * 32 * kConsumerWarps, it.rows * n - 1);
            lse[u] = __ldcg(p.part_lse + slot(x % n) + x / n);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (k + u * 32 * kConsumerWarps < it.rows * n)
                room[k + u * 32 * kConsumerWarps] = lse[u];
    }
    if (!consumer_sync(p, c, sph))
        return false;
    for (int r = warp; r < it.rows; r += kConsumerWarps) {
        float M = -INFINITY, W = 0.f;
        for (int i = lane; i < n; i += 32)
            M = fmaxf(M, room[r * n + i]);
        M = dev::warp_max(M);
        for (int i = lane; i < n; i += 32) {
            const float h = M == -INFINITY ? 0.f : root_weight(room[r * n + i] - M);
            room[r * n + i] = h;
            W += h * h;
        }
        W = dev::warp_sum(W);
        const float root = sqrtf(W);  // (at least 1, or 0 without any weight)
        for (int i = lane; i < n; i += 32)
            room[r * n + i] = W > 0.f ? room[r * n + i] / root : 0.f;
    }
    if (!consumer_sync(p, c, sph))
        return false;
    const int group = tid / LR, col = tid % LR * 4;
    const int ways = max(kGroups / it.rows, 1);           // groups that share a row
    const int sub = group % ways, step = kGroups / ways;
    float *const part = room + (it.rows * n + 3) / 4 * 4 + group * D + col;
    T *const out = reinterpret_cast<T *>(p.out) + ((size_t)it.seq * p.num_q_heads + it.qrow0) * D + col;
    for (int r = group / ways; r < it.rows; r += 2 * step) {
        const int r2 = min(r + step, it.rows - 1);
        float o[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        for (int k0 = sub; k0 < n; k0 += ways * kFlight) {
            float4 v[2][kFlight];
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                const float *src = p.part_o + (size_t)slot(min(k0 + u * ways, n - 1)) * D + col;
                v[0][u] = __ldcg(reinterpret_cast<const float4 *>(src + (size_t)r * D));
                v[1][u] = __ldcg(reinterpret_cast<const float4 *>(src + (size_t)r2 * D));
            }
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                const int k = k0 + u * ways;
                const float w0 = k < n ? room[r * n + k] : 0.f, w1 = k < n ? room[r2 * n + k] : 0.f;
                if (k < n) {
                    o[0][0] = fmaf(w0, w0 * v[0][u].x, o[0][0]);
                    o[0][1] = fmaf(w0, w0 * v[0][u].y, o[0][1]);
                    o[0][2] = fmaf(w0, w0 * v[0][u].z, o[0][2]);
                    o[0][3] = fmaf(w0, w0 * v[0][u].w, o[0][3]);
                    o[1][0] = fmaf(w1, w1 * v[1][u].x, o[1][0]);
                    o[1][1] = fmaf(w1, w1 * v[1][u].y, o[1][1]);
                    o[1][2] = fmaf(w1, w1 * v[1][u].z, o[1][2]);
                    o[1][3] = fmaf(w1, w1 * v[1][u].w, o[1][3]);
                }
            }
        }
        if (ways > 1) {  // (step >= rows: one row for this group)
            *reinterpret_cast<float4 *>(part) = make_float4(o[0][0], o[0][1], o[0][2], o[0][3]);
        } else {
            store4(out + (size_t)r * D, o[0]);
            if (r + step < it.rows)
                store4(out + (size_t)r2 * D, o[1]);
        }
    }
    if (ways > 1) {
        if (!consumer_sync(p, c, sph))
            return false;
        const int r = group / ways;
        if (sub == 0 && r < it.rows) {
            float o[4] = {0.f, 0.f, 0.f, 0.f};
            for (int u = 0; u < ways; ++u) {
                const float4 v = *reinterpret_cast<const float4 *>(part + u * D);
                o[0] += v.x;
                o[1] += v.y;
                o[2] += v.z;
                o[3] += v.w;
            }
            store4(out + (size_t)r * D, o);
        }
    }
    return consumer_sync(p, c, sph);  // the merge rows are read before the next item's come
}

// The same with a row for each thread group and nothing to exchange: rounds of eight
// parts' log2-sum-exps and rows, read at once.  (152 units of 13 rows of 64 dims, each cut
// once: 15.7 us against merge8's 17.5; 104 cut in three: 13.5 against 15.4.)
template <typename T, int D>
__device__ __forceinline__ void merge_few(const DecodeParams &p, const Item &it, int tid)
{
    constexpr int LR = D / 4;
    const int n = it.nparts, col = tid % LR * 4;
    for (int r = tid / LR; r < it.rows; r += 32 * kConsumerWarps / LR) {
        float M = -INFINITY, W = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int k0 = 0; k0 < n; k0 += kFlight) {
            float lse[kFlight];
            float4 v[kFlight];
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                // (the parts' slots: merge8)
                const int k = min(k0 + i, n - 1);
                const int row = (2 * (it.c_first + k) + (k == 0 ? 1 : 0)) * kHeadsPerItem + r;
                lse[i] = __ldcg(p.part_lse + row);
                v[i] = __ldcg(reinterpret_cast<const float4 *>(p.part_o + (size_t)row * D + col));
            }
            float m = M;
#pragma unroll
            for (int i = 0; i < kFlight; ++i)
                m = fmaxf(m, lse[i]);
            const float h = M == -INFINITY ? 0.f : root_weight(M - m);
            M = m;
            W *= h * h;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = h * (h * o[e]);
#pragma unroll
            for (int i = 0; i < kFlight; ++i)
                if (k0 + i < n)
                    add_part(o, W, M, lse[i], v[i]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = W > 0.f ? o[e] / W : 0.f;
        store4(reinterpret_cast<T *>(p.out) + ((size_t)it.seq * p.num_q_heads + it.qrow0 + r) * D + col, o);
    }
}

// Whether merge_few's rounds take less than merge8's two exchanges: up to 16 parts, or 40
// where the rows fill the groups of threads once.  Whole calls, one unit of so many parts,
// bf16, us with merge_few / merge8:
//     parts                  6          10          16          20          32          40
//     128 dims,  1 row   8.5/10.0    8.5/10.0    9.3/10.2   10.5/10.5   10.9/10.4   12.7/11.4
//                4 rows  8.5/9.9     8.6/10.0    9.5/10.9   10.7/11.8   11.2/12.5   12.8/13.6
//                8 rows  9.8/10.8   10.0/11.0   11.6/12.0   13.4/12.8   14.6/13.6   16.9/14.8
//               16 rows 14.3/15.2   15.0/15.8   18.2/17.5   21.3/19.3   24.1/21.2   28.0/24.1
//      64 dims,  1 row   8.9/10.2    8.7/9.9     9.8/10.3   10.5/10.5   11.4/10.7   12.8/10.8
//                8 rows  8.5/10.2    9.1/10.7    9.8/11.6   10.4/12.0   11.5/13.2   12.4/14.1
//               16 rows 10.9/12.7   11.4/13.1   13.1/14.1   14.4/14.8   16.2/16.0   17.6/17.6
// (The full groups, 4 rows of 128 dims and 8 of 64, keep a lead of 1.5 us at 64 parts.)
template <int D>
__device__ __forceinline__ bool few_rounds(const Item &it)
{
    constexpr int kGroups = 128 * kConsumerWarps / D;
    return it.nparts <= (it.rows > kGroups / 2 && it.rows <= kGroups ? 40 : 16);
}

// Count this CTA's part of a split unit; whether it was the last.  `seen`: the counter as
// read before.  As count_partial, but where the counter has this launch's epoch already
// an add takes the place of further exchanges: the parts of one long unit finish together,
// and each round of exchanges lets one of them through (38 parts took 20 us).
__device__ __forceinline__ bool count8(const DecodeParams &p, const Item &it, unsigned long long seen)
{
    unsigned long long *ctr = p.counters + it.c_first;
    unsigned int cnt = 0;
    // (each failed exchange means that another CTA changed the counter: at most nparts)
    while ((unsigned int)(seen >> 32) != p.epoch) {
        const unsigned long long prev = atomicCAS(ctr, seen, ((unsigned long long)p.epoch << 32) | 1ull);
        if (prev == seen) {
            cnt = 1;
            break;
        }
        seen = prev;
    }
    if (cnt == 0)
        cnt = (unsigned int)atomicAdd(ctr, 1ull) + 1u;
    const bool last = cnt == (unsigned int)it.nparts;
    if (last)  // every part is counted: no other CTA touches this counter again
        *reinterpret_cast<volatile unsigned long long *>(ctr) = 0ull;
    return last;
}

// The other part's rows of a unit cut once, when its counter, read as `seen`, says that
// they are there; the counter is then reset for the next launch (count_partial).  -1:
// this part is stored and counted.
__device__ __forceinline__ int other_part(const DecodeParams &p, const Item &it, unsigned long long seen)
{
    if (!it.partial || it.nparts != 2 || seen != (((unsigned long long)p.epoch << 32) | 1ull))
        return -1;
    dev::fence_acq_rel_gpu();  // its rows were released before its count
    *reinterpret_cast<volatile unsigned long long *>(p.counters + it.c_first) = 0ull;
    const int s0 = (2 * it.c_first + 1) * kHeadsPerItem, s1 = 2 * (it.c_first + 1) * kHeadsPerItem;
    return s0 == it.prow0 ? s1 : s0;
}

// End of an item: the barrier before the merge buffers are used again and, for a split
// unit whose part went to its slot, the release, the count and the merge (see
// finish_item).  False on a timeout.
template <typename T, int D>
__device__ __forceinline__ bool finish8(const DecodeParams &p, const Item &it, const CtaState &c, uint32_t &sph,
                                        int warp, int lane, int rows_cap, bool counted,
                                        unsigned long long seen)
{
    if (!consumer_sync(p, c, sph))
        return false;
    if (!it.partial || counted)
        return true;
    if (threadIdx.x == 0) {
        dev::fence_acq_rel_gpu();
        const bool last = count8(p, it, seen);
        if (last)
            dev::fence_acq_rel_gpu();
        *c.merge = last ? 1 : 0;
    }
    if (!consumer_sync(p, c, sph))
        return false;
    if (!*c.merge)
        return true;
    // merge8 needs room for weights and, with few rows, a row per group of threads; a unit of
    // more parts (8 rows of 64 dims: over 223) takes merge_few's rounds, 60000 tokens 33.5 us.
    if (!few_rounds<D>(it) && it.rows * it.nparts + 3 + 4 * 128 <= merge_room(rows_cap, D))
        return merge8<T, D>(p, it, c, sph, warp, lane, c.macc);
    merge_few<T, D>(p, it, warp * 32 + lane);
    return true;
}

template <typename T, int D, int BS, int NT>
__global__ void __launch_bounds__(kThreads8, Cfg8<T, D, BS, NT>::kCtas)
    pa_q8_decode_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ Q8Params q8,
                        const __grid_constant__ CUtensorMap map)
{
    using C = Cfg8<T, D, BS, NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem =
        reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int rows_cap = item_rows_cap(p);
    const SmemLayout lay = make_layout8(C::kStages, C::kStageBytes, C::kBPS, C::kSlots, rows_cap, D, sizeof(T));
    CtaState c = cta_state(smem, lay, C::kStages);
    c.item_empty = c.item_full + C::kSlots;
    c.csync = c.item_empty + C::kSlots;
    uint64_t *const sfull = c.csync + 1;
    // (init_cta knows kItemSlots item slots and no scale barriers)
    if (threadIdx.x < C::kStages)
        dev::mbar_init(dev::smem_addr(&sfull[threadIdx.x]), 1);
    if (threadIdx.x >= kItemSlots && threadIdx.x < C::kSlots) {
        dev::mbar_init(dev::smem_addr(&c.item_full[threadIdx.x]), 1);
        dev::mbar_init(dev::smem_addr(&c.item_empty[threadIdx.x]), kConsumerWarps);
    }
    dev::fence_mbar_init();
    init_cta(p, c, C::kStages);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (warp == kConsumerWarps) {
        Producer8<T, D, BS, NT> pr(p, &map, c, lane);
        walk_balanced<kModePlain>(p, BS, C::kBPS, pr, lane);
        pr.finish();
        return;
    }
    if (warp > kConsumerWarps) {
        ScaleWarp<T, D, BS, NT> sw(p, q8, c, sfull, lane);
        walk_balanced<kModePlain>(p, BS, C::kBPS, sw, lane);
        return;
    }
    // Two merge flags in turn: warp 0 may set the next item's while another warp has yet to
    // read this one's (it cannot be two ahead: the barrier between takes every warp).
    volatile int *merge_now = c.merge;
    volatile int *merge_next = reinterpret_cast<volatile int *>(smem + lay.flag + 16 + 4 * kConsumerWarps);
    uint32_t g = 0;    // stages consumed (same count in every warp)
    uint32_t sph = 0;  // consumer barrier phase
    for (uint32_t n = 0;; ++n) {
        const uint32_t slot = n % C::kSlots;
        if (!warp_wait(p, c, &c.item_full[slot], (n / C::kSlots) & 1u))
            break;
        const Item it = load_item(&c.items[slot]);
        if (it.seq < 0)
            break;
        // A whole unit of at most one stage belongs to one warp, from the query rows to
        // the output, and the warps go on to the next items without meeting (400 sequences
        // of 20 tokens, 8 heads: 39.6 us to 23.9).  With 9 heads or more per kv head there
        // are few such items, and the code for them costs registers that are short.
        const bool alone = NT == 1 && !it.partial && it.j1 - it.j0 <= C::kBPS;
        if (alone && warp != it.rot()) {
            release_item(c, it, slot, warp, lane, 0u);
            g += it.j1 > it.j0 ? 1 : 0;
            if (*c.abort)
                break;
            continue;
        }
        unsigned long long seen = 0;  // thread 0: the split unit's counter
        if (!consume_item8<T, D, BS, NT>(p, c, it, sfull, slot, g, warp, lane, rows_cap, alone, seen))
            break;
        if (alone) {
            if (*c.abort)
                break;
            continue;
        }
        c.merge = merge_now;
        merge_now = merge_next;
        merge_next = c.merge;
        if (threadIdx.x == 0)
            *c.merge = other_part(p, it, seen);
        if (!consumer_sync(p, c, sph))
            break;
        const int other = *c.merge;
        finalize8<T, D>(p, it, c.macc, c.mml, rows_cap, threadIdx.x, other);
        if (!finish8<T, D>(p, it, c, sph, warp, lane, rows_cap, other >= 0, seen))
            break;
        if (*c.abort)
            break;
    }
}

template <typename T, int D, int BS, int NT>
cudaError_t launch_q8_impl(const Q8Launch &L, cudaStream_t stream)
{
    using C = Cfg8<T, D, BS, NT>;
    const DecodeParams &p = L.p;
    void *kern = reinterpret_cast<void *>(&pa_q8_decode_kernel<T, D, BS, NT>);
    const size_t smem =
        make_layout8(C::kStages, C::kStageBytes, C::kBPS, C::kSlots, item_rows_cap(p), D, sizeof(T)).total;
    const size_t smem_max = make_layout8(C::kStages, C::kStageBytes, C::kBPS, C::kSlots, NT * 8, D, sizeof(T)).total;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const int per_sm = cached_occupancy(kern, dev, smem, smem_max, kThreads8);
    if (per_sm <= 0)
        return cudaErrorInvalidConfiguration;
    void *args[] = {const_cast<DecodeParams *>(&L.p), const_cast<Q8Params *>(&L.q8),
                    const_cast<CUtensorMap *>(&L.map)};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(min(per_sm, kMaxCtasPerSm) * L.sm_count));
    cfg.blockDim = dim3(kThreads8);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, kern, args);
}

// Items of at most 8 query rows take one group of the products' 8 columns.
template <typename T, int D, int BS>
cudaError_t launch_q8_rows(const Q8Launch &L, cudaStream_t stream)
{
    return L.p.group <= kNarrowRows ? launch_q8_impl<T, D, BS, 1>(L, stream)
                                    : launch_q8_impl<T, D, BS, 2>(L, stream);
}

template <typename T>
cudaError_t launch_q8_dispatch(const Q8Launch &L, cudaStream_t stream)
{
    if (L.head_dim == 128 && L.block_size == 16)
        return launch_q8_rows<T, 128, 16>(L, stream);
    if (L.head_dim == 128 && L.block_size == 32)
        return launch_q8_rows<T, 128, 32>(L, stream);
    if (L.head_dim == 64 && L.block_size == 16)
        return launch_q8_rows<T, 64, 16>(L, stream);
    if (L.head_dim == 64 && L.block_size == 32)
        return launch_q8_rows<T, 64, 32>(L, stream);
    return cudaErrorInvalidValue;
}

}  // namespace pagedkv
