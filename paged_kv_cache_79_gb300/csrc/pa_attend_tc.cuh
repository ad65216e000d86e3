// pa_attend for fp16 and bf16: tcgen05 with accumulators in TMEM.
//
// An item has two tiles of 128 rows (rows: query tokens times heads of a group) that step
// through the same keys, 128 at a time.  Per CTA, one per SM:
//   warp 8       loader: per tile of keys one TMA copy for each cache block and 128-byte
//                column of K, then one for each block of V, into a ring.  Block ids are read a
//                window of 32 ahead (a read takes longer than a tile when DRAM is busy), an
//                item's first ones when the loader comes to it;
//   warp 10      makes the rows behind the last key that an item sees zeros in V (a weight of
//                0 times what a stale row holds would be NaN where that is NaN);
//   warp 9       products, issued by one lane: S = Q K^T into TMEM (operands in shared
//                memory), O += P V with P read from TMEM;
//   warp 11      walks through the CTA's share, hands the items on to the others and copies
//                Q's rows with TMA;
//   warps 0..3   softmax of the first row tile, warps 4..7 of the second: a thread has a row.
//                It reads its 128 scores from TMEM, writes its probabilities over them as
//                fp16/bf16, and keeps the row's maximum and sum.
// While one row tile's scores are in its softmax, the tensor cores work on the other's.
//
// The running maximum need not be the true one: any base with exponents that stay in range
// gives the same quotient.  So a tile's probabilities are taken by the base at hand while the
// tile's maximum is still being found, and only where a row's maximum has outgrown its base by
// too much (bf16: 2^8), O (in TMEM) is rescaled and the tile's probabilities are taken again.
//
// fp16 has no room below: weights under 2^-14 would lose bits and those under 2^-25 vanish, which
// over a long context adds up.  There the base lies 2^11 below the maximum and may lag by 2^4
// more: weights reach 2^15 (fp16 ends at 2^16), and only those under 2^-25 of the largest lose
// bits, 2^-36 of it at most.  (4096-token prompts of 40 heads 315.6 us; a base 2^7 below and a lag
// of 2^8, with 2^4 less room, 312.5.)
//
// Where an item has one row tile (few query tokens), its tiles of keys go to the two softmax groups
// in turn, each with an output of its own over the same rows, and the first joins them.
//
// Measured (32 / 8 heads of 128, bf16, causal): two prompts of 8192 tokens 723 to 731 us, 1350
// TFLOP/s, 69% of the measured bf16 rate; 1000 tokens behind 95,000 1142 to 1199 us.  64 sequences
// of 1 to 8 tokens over 500 to 8192 keys, 64 / 8 heads: 136 us, 5360 GB/s, 79% of the measured copy.
// Bound by the products (the tensor pipe is busy 70% of the time) and the hand-overs between
// them and the softmax, of which the other row tile covers a part; with few tokens by DRAM.
#pragma once

#include "pa_attend.cuh"

namespace pagedkv {
namespace tc {

constexpr int kThreads = 384;
constexpr int kLoaderWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kTailWarp = 10;
constexpr int kQueryWarp = 11;
constexpr int kTileRows = 128;
constexpr int kKeys = 128;
constexpr int kChunkBytes = kKeys * 128;   // 128 rows of 128 bytes: one column of a tile
// Exponents (log2) that a row's scores may reach over its base before it is taken anew.  (It lies
// kAttendBelow below the maximum; from 2^24 on it rounds to a multiple of up to 8, so by at most 8.)
template <typename T>
constexpr float kRescale = std::is_same<T, __half>::value ? 15.0f : 8.0f;
constexpr float kFar = 1048576.0f;         // bases (log2) from which on products are rounded first
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;            // O of the row tiles, behind their S (128 columns each)

// An item, or a part of one, as the warps need it.  One warp walks through the stream and hands
// the items on through shared memory: each step takes thousands of cycles (64-bit divisions, the
// lengths of the next sequence), which every role would else wait for at every item.
struct alignas(16) Item {
    int s;                // sequence
    int seen;             // keys that the last token sees
    int a, b;             // tiles of keys
    int token0, tokens;   // query tokens (rows of q)
    int head0, heads;     // query heads
    int kv;               // kv head
    int T;                // keys of the sequence
    int own;              // causal: keys that the first token sees (may be below 0)
    int whole;            // all of the item's tiles; 0: partial rows
    int dual;             // one row tile: both softmax groups take its tiles of keys in turn
    int valid;            // 0: no more
    int unused[2];
};
constexpr int kItems = 4;                             // handed on ahead
constexpr int kItemReaders = 8 + 3;                   // warps that read them

template <int D>
struct Smem {
    static constexpr int kChunks = D / 64;
    static constexpr int kTileBytes = kChunks * kChunkBytes;  // 128 rows of Q, K or V
    static constexpr int kStages = D == 128 ? 5 : 10;         // what shared memory holds
    static constexpr int kRing = 2 * kTileBytes;              // behind the two tiles of Q
    static constexpr int kBars = kRing + kStages * kTileBytes;
    static constexpr int kFull = kBars, kEmpty = kFull + 8 * kStages, kRaw = kEmpty + 8 * kStages,
                         kQFull = kRaw + 8 * kStages,
                         kQEmpty = kQFull + 16, kSFull = kQEmpty + 16, kPFull = kSFull + 16, kODone = kPFull + 16,
                         kPair = kODone + 16, kPairFree = kPair + 8, kItemFull = kPairFree + 8, kItemEmpty = kItemFull + 8 * kItems,
                         kDrain = kItemEmpty + 8 * kItems, kTmem = kDrain + 8, kAbort = kTmem + 4, kScratch = kAbort + 4,
                         kSlots = (kScratch + 8 * (kThreads / 32 + 4) + 15) / 16 * 16,
                         kPairRows = kSlots + kItems * (int)sizeof(Item),
                         kEnd = kPairRows + kTileRows * 8;
    static constexpr int kBytes = kEnd + 1024;                // slack to align the base
    static_assert(kBytes <= 232448, "one CTA's shared memory");
};

// ---- tcgen05 -------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t slot)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t base)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(kTmemCols) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// `bar` is arrived at when every product issued so far by this thread has completed.
__device__ __forceinline__ void commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// D (+)= A B, operands in shared memory; and with A in TMEM.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// 32 columns of this warp's 32 rows, a row per lane.
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t addr)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14,"
        " %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14,"
        " %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
// The loads so far have arrived, among them r (named so that no use of it moves ahead).
__device__ __forceinline__ void wait_ld(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                   "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])::"memory");
}

// N consecutive words of a row, 32 bytes (whole sectors) at a time where the address allows it.
template <int N>
__device__ __forceinline__ void store_words(void *dst, const uint32_t (&w)[N], bool wide)
{
    if (wide) {
#pragma unroll
        for (int i = 0; i < N; i += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                             static_cast<uint32_t *>(dst) + i),
                         "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]),
                         "r"(w[i + 6]), "r"(w[i + 7])
                         : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            static_cast<uint4 *>(dst)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
}

// Two fp32 operations at a time, and the larger of three.
__device__ __forceinline__ unsigned long long bits(float2 x)
{
    return (unsigned long long)__float_as_uint(x.y) << 32 | __float_as_uint(x.x);
}
__device__ __forceinline__ float2 pair(unsigned long long x)
{
    return make_float2(__uint_as_float((uint32_t)x), __uint_as_float((uint32_t)(x >> 32)));
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
    return pair(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
    return pair(d);
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// One lane of the warp (the same each time), in a form that leaves the code around it uniform.
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// Shared-memory operand: 128-byte swizzle.  Rows of 128 bytes along K (Q and K: K-major):
// groups of 8 rows `sbo` apart.  Rows of 128 bytes along N (V): groups of 8 keys `sbo` apart,
// the next 64 columns `lbo` on.  (A product takes all of K's rows, evenly spaced, so a block's
// columns lie a whole tile apart; of V it takes 16 keys at a time, so blocks may stay whole.)
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lbo, uint32_t sbo)
{
    return (uint64_t)((addr >> 4) & 0x3fff) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 | 1ull << 46 |
           2ull << 61;
}
// fp32 accumulators, 16-bit operands (format 0: fp16, 1: bf16), 128 rows, n columns.
__host__ __device__ constexpr uint32_t instruction(uint32_t format, uint32_t n, bool b_along_n)
{
    return 1u << 4 | format << 7 | format << 10 | (b_along_n ? 1u << 16 : 0u) | (n >> 3) << 17 |
           (uint32_t)(kTileRows >> 4) << 24;
}

__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

template <typename T, int D, int B>
__global__ void __launch_bounds__(kThreads, 1)
    attend_kernel(const __grid_constant__ AttendParams p, const __grid_constant__ CUtensorMap map_q,
                  const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v)
{
    using S = Smem<D>;
    using Walk = AttendWalk<kKeys>;
    constexpr int kChunks = S::kChunks;
    constexpr int kBlocks = kKeys / B;  // cache blocks per tile of keys
    constexpr uint32_t kFormat = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t smem = (dev::smem_addr(smem_raw) + 1023u) & ~1023u;
    unsigned char *const smem_ptr = smem_raw + (smem - dev::smem_addr(smem_raw));
    volatile int *const abort = reinterpret_cast<volatile int *>(smem_ptr + S::kAbort);
    auto &scratch = *reinterpret_cast<long long(*)[kThreads / 32 + 4]>(smem_ptr + S::kScratch);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        dev::tma_prefetch_desc(&map_q);
        dev::tma_prefetch_desc(&map_k);
        dev::tma_prefetch_desc(&map_v);
        for (int i = 0; i < S::kStages; ++i) {
            dev::mbar_init(smem + S::kFull + 8 * i, 1);
            dev::mbar_init(smem + S::kEmpty + 8 * i, 1);
            dev::mbar_init(smem + S::kRaw + 8 * i, 1);
        }
        for (int t = 0; t < 2; ++t) {
            dev::mbar_init(smem + S::kQFull + 8 * t, 1);
            dev::mbar_init(smem + S::kQEmpty + 8 * t, 1);
            dev::mbar_init(smem + S::kSFull + 8 * t, 1);
            dev::mbar_init(smem + S::kPFull + 8 * t, kTileRows / 32);  // a warp each
            dev::mbar_init(smem + S::kODone + 8 * t, 1);
        }
        dev::mbar_init(smem + S::kPair, kTileRows / 32);
        dev::mbar_init(smem + S::kPairFree, kTileRows / 32);
        for (int i = 0; i < kItems; ++i) {
            dev::mbar_init(smem + S::kItemFull + 8 * i, 1);
            dev::mbar_init(smem + S::kItemEmpty + 8 * i, kItemReaders);
        }
        dev::mbar_init(smem + S::kDrain, 1);
        *abort = 0;
        dev::fence_mbar_init();
    }
    dev::grid_dependency_wait();
    dev::grid_launch_dependents();
    Walk walk(p);
    if (!walk.template begin<kThreads>(scratch))
        return;
    if (warp == kMmaWarp)
        tmem_alloc(smem + S::kTmem);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem_ptr + S::kTmem);
    const int half_tokens = p.tokens_per_item / 2;  // of a row tile

    // A bounded wait; false: this CTA gives up.
    auto wait = [&](uint32_t bar, uint32_t parity, unsigned int flag) {
        const int r = dev::mbar_wait_abortable(bar, parity, p.wait_ns, abort);
        if (r == 0) {
            atomicOr(p.errors, flag);
            *abort = 1;
        }
        return r > 0;
    };
    // The same by a whole warp, all of whose lanes go on or none.
    auto wait_all = [&](uint32_t bar, uint32_t parity, unsigned int flag) {
        return __all_sync(0xffffffffu, wait(bar, parity, flag)) != 0;
    };

    // The next item for a warp that reads them in turn (`turn`: how many it has read).
    Item *const slots = reinterpret_cast<Item *>(smem_ptr + S::kSlots);
    auto next_item = [&](Item &it, uint32_t &turn) {
        const uint32_t i = turn % kItems;
        if (!wait_all(smem + S::kItemFull + 8 * i, turn / kItems & 1, PA_DEVERR_TIMEOUT_FULL))
            return false;
        it = slots[i];
        __syncwarp();
        if (lane == 0)
            dev::mbar_arrive(smem + S::kItemEmpty + 8 * i);
        ++turn;
        return it.valid != 0;
    };

    // The softmax warps hold 128 scores a thread: 168 registers each at launch (three warps per
    // scheduler) become 2 x 200 and 104.
    if (warp >= kLoaderWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        if (warp == kLoaderWarp) {
            uint32_t stage = 0, round = 0;                // of the ring
            uint32_t filled = 0, raw = 0, raw_round = 0;  // bits: stages filled, filled with a tail, its parity
            bool ok = true;
            // The blocks of 32 / kBlocks tiles from `tile` on, one per lane (past the last that is seen, or
            // outside the pool: past the pool's end, where a copy brings zeros).
            constexpr int kWindow = 32 / kBlocks;
            auto window = [&](const Item &it, int tile) {
                const int j = tile * kBlocks + lane;
                int id = -1;
                if (j < min((int)(((unsigned int)it.seen + (B - 1)) / B), it.b * kBlocks))
                    id = p.block_tables[(size_t)it.s * p.max_blocks + j];
                return id >= 0 && id < p.num_blocks ? id : p.num_blocks;
            };
            Item it;
            uint32_t turn = 0;
            while (ok && next_item(it, turn)) {
                if (it.a == it.b)
                    continue;
                int id = window(it, it.a), id_next = window(it, it.a + kWindow);
                const int kv_head = __shfl_sync(0xffffffffu, it.kv, 0);
                int slot = 0;  // of the window
                for (int tile = it.a; tile < it.b && ok; ++tile) {
                    int ids[kBlocks];
#pragma unroll
                    for (int i = 0; i < kBlocks; ++i)
                        ids[i] = __shfl_sync(0xffffffffu, id, slot * kBlocks + i);
                    if (++slot == kWindow) {
                        slot = 0;
                        id = id_next;
                        id_next = window(it, tile + 1 + kWindow);
                    }
                    const int keys = __shfl_sync(0xffffffffu, min(it.seen - tile * kKeys, kKeys), 0);  // of this tile
                    const int copies = (keys + B - 1) / B;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        ok = wait_all(smem + S::kEmpty + 8 * stage, round ^ 1, PA_DEVERR_TIMEOUT_EMPTY);
                        if (!ok)
                            break;
                        // V with rows behind the last key goes to the tail warp first
                        const bool tail = kv == 1 && keys < kKeys;
                        const uint32_t at = smem + S::kRing + stage * S::kTileBytes;
                        const uint32_t bar = smem + (tail ? S::kRaw : S::kFull) + 8 * stage;
                        if (elect_one()) {
                            dev::mbar_arrive_expect_tx(bar, (uint32_t)(copies * B) * 128u * kChunks);
#pragma unroll
                            for (int i = 0; i < kBlocks; ++i) {
                                if (i >= copies)
                                    break;
                                if (kv == 1) {
                                    dev::tma_load_4d(at + i * (B * 128 * kChunks), &map_v, 0, ids[i] * B, 0, kv_head, bar);
                                } else {
#pragma unroll
                                    for (int c = 0; c < kChunks; ++c)
                                        dev::tma_load_4d(at + c * kChunkBytes + i * (B * 128), &map_k, 0, ids[i] * B, c,
                                                         kv_head, bar);
                                }
                            }
                        }
                        __syncwarp();
                        const uint32_t bit = 1u << stage;
                        filled |= bit;
                        raw = tail ? raw | bit : raw & ~bit;
                        raw_round ^= tail ? bit : 0;
                        if (++stage == S::kStages) {
                            stage = 0;
                            round ^= 1;
                        }
                    }
                }
            }
            // What is in flight lands before the CTA ends.  (Always waited for: whether another warp will
            // have given up, and so not have waited for it, is not known here.)
            for (uint32_t i = 0; i < S::kStages; ++i) {
                if (!(filled >> i & 1))
                    continue;
                // (stages before `stage` were filled in this round, the others in the one before)
                const uint32_t parity = raw >> i & 1 ? (raw_round >> i & 1) ^ 1 : i < stage ? round : round ^ 1;
                dev::mbar_wait(smem + (raw >> i & 1 ? S::kRaw : S::kFull) + 8 * i, parity, kWaitTimeoutNs);
            }
        } else if (warp == kQueryWarp) {
            uint32_t q_round = 0, q_used = 0;  // bit t: row tile t
            uint32_t turn = 0;
            bool ok = true;
            const uint32_t q_bytes = (uint32_t)(half_tokens * p.heads_per_item) * 128u * kChunks;
            auto hand_on = [&](const Item &it) {
                const uint32_t i = turn % kItems;
                ok = wait_all(smem + S::kItemEmpty + 8 * i, (turn / kItems & 1) ^ 1, PA_DEVERR_TIMEOUT_EMPTY);
                if (ok && lane == 0) {
                    slots[i] = it;
                    dev::mbar_arrive(smem + S::kItemFull + 8 * i);
                }
                __syncwarp();
                ++turn;
            };
            do {
                Item it;
                if (!walk.part(it.a, it.b))
                    continue;
                const auto rows = Walk::rows_of(p, walk.it);
                it.s = walk.it.s;
                it.seen = walk.it.seen;
                it.token0 = rows.token0;
                it.tokens = rows.tokens;
                it.head0 = rows.head0;
                it.heads = rows.heads;
                it.kv = rows.kv;
                it.T = walk.it.T;
                it.own = walk.it.T - walk.it.n + walk.it.j * p.tokens_per_item + 1;
                it.whole = it.a == 0 && it.b == walk.it.tiles;
                it.dual = rows.tokens <= half_tokens && it.b - it.a > 1;
                it.valid = 1;
                hand_on(it);
                if (it.a == it.b)
                    continue;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (!ok || (t == 1 && rows.tokens <= half_tokens && !it.dual))
                        break;
                    ok = wait_all(smem + S::kQEmpty + 8 * t, (q_round >> t & 1) ^ 1, PA_DEVERR_TIMEOUT_EMPTY);
                    if (!ok)
                        break;
                    if (elect_one()) {
                        const uint32_t bar = smem + S::kQFull + 8 * t;
                        dev::mbar_arrive_expect_tx(bar, q_bytes);
#pragma unroll
                        for (int c = 0; c < kChunks; ++c)
                            dev::tma_load_4d(smem + t * S::kTileBytes + c * kChunkBytes, &map_q, 0, rows.head0,
                                             rows.token0 + (it.dual ? 0 : t * half_tokens), c, bar);
                    }
                    __syncwarp();
                    q_round ^= 1u << t;
                    q_used |= 1u << t;
                }
            } while (ok && walk.next() && walk.inside());
            if (ok) {
                Item none = {};
                hand_on(none);
            }
            for (int t = 0; t < 2; ++t)  // (as the loader)
                if (q_used >> t & 1)
                    dev::mbar_wait(smem + S::kQFull + 8 * t, (q_round >> t & 1) ^ 1, kWaitTimeoutNs);
        } else if (warp == kTailWarp) {
            // V's rows behind the last key an item sees become zeros, once they have landed.
            uint32_t stage = 0, raw_round = 0, turn = 0;
            bool ok = true;
            Item it;
            while (ok && next_item(it, turn)) {
                if (it.a == it.b)
                    continue;
                const int keys = it.seen - (it.b - 1) * kKeys;  // of the last tile
                stage = (stage + 2 * (uint32_t)(it.b - it.a) - 1) % S::kStages;  // its V
                if (keys < kKeys) {
                    ok = wait_all(smem + S::kRaw + 8 * stage, raw_round >> stage & 1, PA_DEVERR_TIMEOUT_FULL);
                    if (!ok)
                        break;
                    raw_round ^= 1u << stage;
                    constexpr int kVecs = D / 8;
                    for (int i = keys * kVecs + lane; i < kKeys * kVecs; i += 32) {
                        const int r = i / kVecs, x = i % kVecs;
                        *reinterpret_cast<uint4 *>(smem_ptr + S::kRing + stage * S::kTileBytes + r / B * (B * 128 * kChunks) +
                                                   x / 8 * (B * 128) + r % B * 128 + (((x % 8) ^ (r & 7)) << 4)) =
                            make_uint4(0, 0, 0, 0);
                    }
                    fence_async_proxy();
                    __syncwarp();
                    if (lane == 0)
                        dev::mbar_arrive(smem + S::kFull + 8 * stage);
                    __syncwarp();
                }
                if (++stage == S::kStages)
                    stage = 0;
            }
        } else if (warp == kMmaWarp) {
            // The whole warp goes through the loop, so that addresses and descriptors stay in uniform
            // registers; one lane issues.  (With one thread alone in the loop each product took 75
            // cycles to issue, more than the 64 it takes to run.)
            constexpr uint32_t kScores = instruction(kFormat, kKeys, false);
            constexpr uint32_t kOutput = instruction(kFormat, D, true);
            // (Scalars only: an array indexed by the row tile would live in local memory, and each wait
            // would cost hundreds of cycles more.)
            uint32_t q_round = 0, p_round = 0;  // bit t: parity of row tile t
            uint32_t fills = 0;                 // of the ring, before this item: its K and V in turn
            bool ok = true;
            const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0);
            auto full = [&](uint32_t f) {
                return wait_all(smem + S::kFull + 8 * (f % S::kStages), f / S::kStages & 1, PA_DEVERR_TIMEOUT_FULL);
            };
            // S of row tile t from fill f
            auto scores = [&](int t, uint32_t f, bool last_keys, bool release) {
                const uint32_t stage = f % S::kStages;
                if (elect_one()) {
                    const uint64_t q = operand(smem + t * S::kTileBytes, 16, 1024);
                    const uint64_t k0 = operand(smem + S::kRing + stage * S::kTileBytes, 16, 1024);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = ((k / 4) * kChunkBytes + (k % 4) * 32) >> 4;
                        mma_ss(base + t * kKeys, q + off, k0 + off, kScores, k > 0);
                    }
                    commit(smem + S::kSFull + 8 * t);
                    if (last_keys)
                        commit(smem + S::kQEmpty + 8 * t);
                    if (release)
                        commit(smem + S::kEmpty + 8 * stage);
                }
                __syncwarp();
            };
            // O of row tile t, once its probabilities are there, from fill f
            auto output = [&](int t, uint32_t f, bool first, bool last_keys, bool release) {
                if (!wait_all(smem + S::kPFull + 8 * t, p_round >> t & 1, PA_DEVERR_TIMEOUT_FULL))
                    return false;
                p_round ^= 1u << t;
                fence_after();
                const uint32_t stage = f % S::kStages;
                if (elect_one()) {
                    const uint64_t v = operand(smem + S::kRing + stage * S::kTileBytes, B * 128, 1024);
                    mma_ts(base + kColO + t * D, base + t * kKeys, v, kOutput, !first);
#pragma unroll
                    for (int k = 1; k < kKeys / 16; ++k) {
                        const uint32_t off = (k * 16 / B * (B * 128 * kChunks) + k * 16 % B * 128) >> 4;
                        mma_ts(base + kColO + t * D, base + t * kKeys + 8 * k, v + off, kOutput, true);
                    }
                    if (last_keys)
                        commit(smem + S::kODone + 8 * t);
                    if (release)
                        commit(smem + S::kEmpty + 8 * stage);
                }
                __syncwarp();
                return true;
            };
            auto queries = [&](int t) {
                const bool r = wait_all(smem + S::kQFull + 8 * t, q_round >> t & 1, PA_DEVERR_TIMEOUT_FULL);
                q_round ^= 1u << t;
                return r;
            };
            Item it;
            uint32_t turn = 0;
            while (ok && next_item(it, turn)) {
                const bool two = __shfl_sync(0xffffffffu, it.tokens > half_tokens ? 1 : 0, 0) != 0;
                const bool dual = __shfl_sync(0xffffffffu, it.dual, 0) != 0;
                const int n = __shfl_sync(0xffffffffu, it.b - it.a, 0);
                if (n == 0)
                    continue;
                if (dual) {
                    // tile j is row tile j % 2's; K of tile j is fill 2 j, V fill 2 j + 1
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        ok = ok && full(fills + 2 * t) && queries(t);
                        if (ok)
                            scores(t, fills + 2 * t, t + 2 >= n, true);
                    }
                    for (int j = 0; j < n && ok; j += 2) {
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (!ok || j + t >= n)
                                break;
                            const uint32_t f = fills + 2 * (j + t);
                            const bool more = j + t + 2 < n;
                            ok = full(f + 1) && output(t, f + 1, j == 0, !more, true);
                            if (ok && more) {
                                ok = full(f + 4);
                                if (ok)
                                    scores(t, f + 4, j + t + 4 >= n, true);
                            }
                        }
                    }
                } else {
                    ok = full(fills);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (!ok || (t == 1 && !two))
                            break;
                        ok = queries(t);
                        if (ok)
                            scores(t, fills, n == 1, t == 1 || !two);
                    }
                    for (int j = 0; j < n && ok; ++j) {
                        const uint32_t f = fills + 2 * j;
                        const bool more = j + 1 < n;
                        ok = full(f + 1);
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (!ok || (t == 1 && !two))
                                break;
                            ok = output(t, f + 1, j == 0, !more, t == 1 || !two);
                            if (!ok || !more)
                                continue;
                            if (t == 0)
                                ok = full(f + 2);
                            if (ok)
                                scores(t, f + 2, j + 2 == n, t == 1 || !two);
                        }
                    }
                }
                fills += 2 * n;
            }
            // every product has completed before the CTA gives its memory back
            if (elect_one())
                commit(smem + S::kDrain);
            __syncwarp();
            dev::mbar_wait(smem + S::kDrain, 0, kWaitTimeoutNs);
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        const int t = warp >> 2;              // row tile
        const int r = tid & (kTileRows - 1);  // row of it: this thread's
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t s_at = tmem + lanes + t * kKeys, o_at = tmem + lanes + kColO + t * D;
        uint32_t steps = 0, parts = 0;
        uint32_t o1_round = 0, pair_round = 0, free_round = 0;
        bool lent = false;
        float2 *const pair_rows = reinterpret_cast<float2 *>(smem_ptr + S::kPairRows);
        bool ok = true;
        const int tok = r / p.heads_per_item, head = r - tok * p.heads_per_item;
        const bool wide = ((reinterpret_cast<uintptr_t>(p.out) | reinterpret_cast<uintptr_t>(p.part_o)) & 31) == 0;
        Item it;
        uint32_t turn = 0;
        while (ok && next_item(it, turn)) {
            const bool any = it.b > it.a, dual = it.dual != 0;
            const uint32_t o1_now = o1_round;  // parity of the second row tile's output
            if (any && (dual || it.tokens > half_tokens))
                o1_round ^= 1;
            if (!dual && t * half_tokens >= it.tokens)
                continue;
            if (lent) {  // the other group has read the output that this one left it
                ok = wait_all(smem + S::kPairFree, free_round, PA_DEVERR_TIMEOUT_FULL);
                if (!ok)
                    break;
                free_round ^= 1;
                lent = false;
            }
            const int row0 = dual ? 0 : t * half_tokens;  // first token of the row tile
            const int step = dual ? 2 : 1, a = it.a + (dual ? t : 0), b = it.b;
            const int my_tok = row0 + tok;  // of the item
            const bool mine = tok < half_tokens && my_tok < it.tokens && head < it.heads;
            const size_t row = (size_t)(it.token0 + my_tok) * p.num_q_heads + it.head0 + head;
            // keys that this row sees, and that every row of the tile sees
            int limit = it.T, common = it.T;
            if (p.causal) {  // (rows behind the item's tokens may pass 2^31)
                limit = (int)min(max((long long)it.own + my_tok, 0ll), (long long)it.T);
                common = (int)min(max((long long)it.own + row0, 0ll), (long long)it.T);
            }
            float m = -INFINITY, l = 0.f;  // the base in use, the sum
            bool far = false;
            for (int tile = a; tile < b; tile += step) {
                ok = wait_all(smem + S::kSFull + 8 * t, steps & 1, PA_DEVERR_TIMEOUT_FULL);
                if (!ok)
                    break;
                ++steps;
                fence_after();
                const int key0 = tile * kKeys;
                const bool masked = common - key0 < kKeys;
                // Exponents of 32 columns: x = s * scale - base, -inf where the key is hidden; their
                // maximum.  `far`: the product is rounded first.  Behind a large base the exact one
                // would differ from it by the product's rounding error, which may be large itself.
                // `plain`, known at compile time: neither hidden keys nor `far` (branches would part the
                // code that the scheduler can interleave).
                auto exponents = [&](auto plain, const uint32_t (&s)[32], int c, float base, bool far, float2 (&x)[16],
                                     float top) {
                    if (!plain && far) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            x[i] = make_float2(__fadd_rn(__fmul_rn(__uint_as_float(s[2 * i]), p.scale_log2), -base),
                                               __fadd_rn(__fmul_rn(__uint_as_float(s[2 * i + 1]), p.scale_log2), -base));
                    } else {
                        const float2 scale2 = make_float2(p.scale_log2, p.scale_log2), base2 = make_float2(-base, -base);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            x[i] = fma2(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), scale2, base2);
                    }
                    if (!plain && masked) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            x[i].x = key0 + 32 * c + 2 * i < limit ? x[i].x : -INFINITY;
                            x[i].y = key0 + 32 * c + 2 * i + 1 < limit ? x[i].y : -INFINITY;
                        }
                    }
                    float top2 = x[0].x;
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        top = max3(top, x[i].x, x[i].y);
                        top2 = max3(top2, x[i + 1].x, x[i + 1].y);
                    }
                    return fmaxf(top, top2);
                };
                // The base follows the row's maximum, this tile's included.
                auto raise = [&]() {
                    const float had = m + kAttendBelow<T>;
                    float top = had;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t s[32];
                        float2 x[16];
                        tmem_ld32(s, s_at + 32 * c);
                        wait_ld(s);
                        top = exponents(std::false_type(), s, c, 0.f, true, x, top);
                    }
                    top = top > had ? top - kAttendBelow<T> : m;
                    const float f = top == -INFINITY ? 1.f : exp2f(m - top);
                    m = top;
                    far = __any_sync(0xffffffffu, mine && fabsf(m) > kFar && m != -INFINITY);
                    return f;
                };
                if (tile == a)
                    raise();
                // The probabilities by a base, their sum, and the largest exponent.
                uint32_t w[64];
                float2 sum, sum2;
                auto probabilities = [&](auto plain) {
                    const float base = m == -INFINITY ? 0.f : m;
                    float top = -INFINITY;
                    sum = sum2 = make_float2(0.f, 0.f);
                    uint32_t s[2][32];
                    tmem_ld32(s[0], s_at);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        wait_ld(s[c & 1]);
                        if (c < 3)
                            tmem_ld32(s[(c + 1) & 1], s_at + 32 * (c + 1));
                        float2 x[16];
                        top = exponents(plain, s[c & 1], c, base, far, x, top);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            x[i].x = dev::ex2(x[i].x);
                            x[i].y = dev::ex2(x[i].y);
                            if (i & 1)
                                sum2 = add2(sum2, x[i]);
                            else
                                sum = add2(sum, x[i]);
                            w[16 * c + i] = dev::Mma<T>::pack(x[i].x, x[i].y);
                        }
                    }
                    return top;
                };
                // By the base at hand; where that has fallen behind, once more by the maximum.
                const float top = masked || far ? probabilities(std::false_type()) : probabilities(std::true_type());
                // (Rows that are not the item's have no vote: they hold other queries or what an earlier
                // kernel left, and a new base rounds every row of the warp differently.)
                if (__any_sync(0xffffffffu, mine && top > (m == -INFINITY ? -INFINITY : kRescale<T>))) {
                    // O is at rest: the scores of this tile came after the product before it
                    const float f = raise();
                    l *= f;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(o, o_at + c);
                        wait_ld(o);
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                        tmem_st32(o_at + c, o);
                    }
                    probabilities(std::false_type());
                }
                l += (sum.x + sum2.x) + (sum.y + sum2.y);
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    tmem_st32(s_at + 32 * c, *reinterpret_cast<const uint32_t(*)[32]>(w + 32 * c));
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0)
                    dev::mbar_arrive(smem + S::kPFull + 8 * t);
            }
            if (!ok)
                break;
            const bool whole = it.whole != 0;
            if (dual && t == 1) {
                // the first group joins the two: it has the same rows, and reads this one's output
                ++parts;
                pair_rows[r] = make_float2(m, l);
                __syncwarp();
                if (lane == 0)
                    dev::mbar_arrive(smem + S::kPair);
                lent = true;
                continue;
            }
            float f0 = 1.f, f1 = 0.f;
            if (any) {
                ok = wait_all(smem + S::kODone + 8 * t, parts & 1, PA_DEVERR_TIMEOUT_FULL);
                if (ok && dual)
                    ok = wait_all(smem + S::kODone + 8, o1_now, PA_DEVERR_TIMEOUT_FULL) &&
                         wait_all(smem + S::kPair, pair_round, PA_DEVERR_TIMEOUT_FULL);
                if (!ok)
                    break;
                ++parts;
                fence_after();
                if (dual) {
                    pair_round ^= 1;
                    const float2 other = pair_rows[r];
                    const float top = fmaxf(m, other.x), ref = top == -INFINITY ? 0.f : top;
                    f0 = exp2f(m - ref);
                    f1 = exp2f(other.x - ref);
                    m = top;
                    l = l * f0 + other.y * f1;
                }
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const size_t part = attend_part_row(p, blockIdx.x, it.a > 0 ? 0 : 1) + my_tok * p.heads_per_item + head;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                if (any) {
                    tmem_ld32(o, o_at + c);
                    wait_ld(o);
                    if (dual) {
                        uint32_t o1[32];
                        tmem_ld32(o1, o_at + D + c);
                        wait_ld(o1);
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            o[k] = __float_as_uint(__uint_as_float(o[k]) * f0 + __uint_as_float(o1[k]) * f1);
                    }
                }
                if (mine && whole) {
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        w[k] = any ? dev::Mma<T>::pack(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv)
                                   : 0u;
                    store_words(static_cast<T *>(p.out) + row * D + c, w, wide);
                } else if (mine) {
                    store_words(p.part_o + part * D + c, o, wide);
                }
                __syncwarp();
            }
            fence_before();  // O has been read before the next item's first probabilities are announced
            if (dual) {
                __syncwarp();
                if (lane == 0)
                    dev::mbar_arrive(smem + S::kPairFree);
            }
            if (mine && whole && p.lse)
                p.lse[row] = attend_lse<T>(m, l);
            if (mine && !whole)
                p.part_ml[part] = make_float2(m, l);
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kMmaWarp)
        tmem_dealloc(tmem);
}

template <typename T, int D, int B>
cudaError_t launch(const AttendLaunch &L, cudaStream_t stream)
{
    int device = 0;
    const cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess)
        return e;
    const size_t smem = Smem<D>::kBytes;
    if (cached_occupancy(reinterpret_cast<void *>(attend_kernel<T, D, B>), device, smem, smem, kThreads) <= 0)
        return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)L.ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attend_kernel<T, D, B>, L.p, L.map_q, L.map_k, L.map_v);
}

template <typename T>
cudaError_t launch_type(const AttendLaunch &L, cudaStream_t stream)
{
    if (L.head_dim == 64)
        return L.p.block_size == 16 ? launch<T, 64, 16>(L, stream) : launch<T, 64, 32>(L, stream);
    return L.p.block_size == 16 ? launch<T, 128, 16>(L, stream) : launch<T, 128, 32>(L, stream);
}

}  // namespace tc
}  // namespace pagedkv
