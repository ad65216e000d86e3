// Block tables that go on from rows of older ones, on the GPU: samples of a prompt, beams,
// finished requests.  The device counterpart of the host allocator's fork, copy-on-write and
// free (CSDN tutorial "PagedAttention实战" §5.1 clone_sequence; "Efficient Memory Management
// for LLM Serving with PagedAttention", azimuth.plus summary, section "Memory sharing").
//
// extra[b] counts block b's references beyond the first.  An old row with c children gives
// each of its full blocks c - 1 more references (c = 0: one less), so the rows of c = 1, most
// of a beam search's, change nothing.  A block whose count passes below 0 has lost its last
// reference; integer atomics leave the same counts whatever their order, and the freed blocks
// are collected by one ordered pass over the counts, so the free list does not depend on it
// either.
//
// Two launches.  The first runs over the whole GPU: it writes the new rows, adds to the
// counts, and marks the children that need a copy of a half-filled last block.  The second, a
// cluster, collects the freed blocks, hands fresh ones to the marked children in order, and
// takes the refused ones back.  Bound by latency: the second needs the counts that the first
// has finished.
// Measured: 16 prompts to 128 samples 8.6 us, 256 beams with a pool of 80,000 blocks 11.6, 1001 rows
// with a pool of 200,000 17.8 (30.3 with the counts scanned 1024 at a time and one CTA handing out
// the copies).
#include <cooperative_groups.h>

#include <climits>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pagedkv {

namespace {

constexpr int kRowThreads = 256;
constexpr int kRowEntries = 1024;  // entries of a row per CTA of the first launch
constexpr int kEndThreads = 1024;
constexpr int kEndCtas = 8;
enum { kEmpty = 0, kContinues = 1, kWantsCopy = 2, kRefused = -1 };

struct Row {
    int len;     // tokens, clamped to the table
    int blocks;
    bool half;   // the last block is not full
};
__device__ __forceinline__ Row row_of(const ForkParams &p, int r)
{
    Row x;
    const long long cap = (long long)p.max_blocks * p.block_size;
    x.len = (int)min((long long)max(p.context_lens[r], 0), cap);
    x.blocks = (int)(((unsigned int)x.len + (unsigned int)(p.block_size - 1)) / (unsigned int)p.block_size);
    x.half = x.len % p.block_size != 0;
    return x;
}

__device__ __forceinline__ void add_refs(const ForkParams &p, int block, int n)
{
    if (block >= 0 && block < p.num_blocks)
        atomicAdd(p.extra + block, n);
}

// CTA (i, c): entries [c kRowEntries, ..) of new row i and of old row i.
__global__ void __launch_bounds__(kRowThreads) fork_rows_kernel(const __grid_constant__ ForkParams p)
{
    dev::grid_dependency_wait();
    dev::grid_launch_dependents();
    const int tid = threadIdx.x;
    const int i = blockIdx.x;
    const int j0 = blockIdx.y * kRowEntries;
    const int j1 = min(p.max_blocks - j0, kRowEntries) + j0;
    if (i < p.children) {
        const int parent = p.parents[i];
        const bool real = parent >= 0 && parent < p.rows;
        Row row = {0, 0, false};
        if (real)
            row = row_of(p, parent);
        const int32_t *src = p.tables_in + (size_t)(real ? parent : 0) * p.max_blocks;
        int32_t *dst = p.tables_out + (size_t)i * p.max_blocks;
        for (int j = j0 + tid; j < j1; j += kRowThreads)
            dst[j] = j < row.blocks ? src[j] : -1;
    }
    // One look through the parents: whether a child before this one keeps the half-filled block,
    // and how many children old row i has.
    const int parent = i < p.children ? p.parents[i] : -1;
    int kids = 0, earlier = 0;
    if (j0 == 0 || i < p.rows)
#pragma unroll 4
        for (int k = tid; k < p.children; k += kRowThreads) {
            const int x = p.parents[k];
            kids += x == i ? 1 : 0;
            earlier |= k < i && x == parent ? 1 : 0;
        }
    __shared__ int s_kids;
    if (tid == 0)
        s_kids = 0;
    earlier = __syncthreads_or(earlier);
    kids = __reduce_add_sync(0xffffffffu, kids);
    if ((tid & 31) == 0 && kids)
        atomicAdd(&s_kids, kids);
    __syncthreads();
    kids = s_kids;
    if (tid == 0 && j0 == 0 && i < p.children) {
        const bool real = parent >= 0 && parent < p.rows;
        p.granted[i] = !real ? kEmpty : earlier && row_of(p, parent).half ? kWantsCopy : kContinues;
    }
    if (i < p.rows && kids != 1) {
        const Row row = row_of(p, i);
        const int32_t *src = p.tables_in + (size_t)i * p.max_blocks;
        const int full = row.blocks - (row.half ? 1 : 0);
        for (int j = j0 + tid; j < min(j1, row.blocks); j += kRowThreads)
            if (j < full || kids == 0)
                add_refs(p, src[j], kids - 1);
    }
}

// Exclusive sums of x over the CTA's threads; *total: all of them.
__device__ __forceinline__ int sum_before(int x, int *total, int (&part)[32])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int in = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, in, o);
        if (lane >= o)
            in += y;
    }
    __syncthreads();  // the previous sums have been read
    if (lane == 31)
        part[warp] = in;
    __syncthreads();
    const int own = part[lane];
    int w = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o)
            w += y;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    return __shfl_sync(0xffffffffu, w - own, warp) + in - x;
}

// A thread goes through kOwn consecutive blocks at a time, so that the ascending order of the
// blocks is the order of the threads and one sum over the CTA places them all.
constexpr int kOwn = 32;
__global__ void __launch_bounds__(kEndThreads) fork_end_kernel(const __grid_constant__ ForkParams p)
{
    namespace cg = cooperative_groups;
    __shared__ int part[32];
    __shared__ int freed, wanted_here;
    cg::cluster_group cluster = cg::this_cluster();
    dev::grid_dependency_wait();
    dev::grid_launch_dependents();
    const int tid = threadIdx.x;
    const int rank = (int)cluster.block_rank();
    const int had = min(max(*p.num_free, 0), p.num_blocks);

    // The blocks that lost their last reference, in ascending order; each CTA a range of blocks, a
    // multiple of kOwn long, each thread kOwn of them as a mask of bits.
    const long long share =
        ((long long)p.num_blocks + kEndCtas * kOwn - 1) / (kEndCtas * kOwn) * kOwn;
    const long long b0 = min(rank * share, (long long)p.num_blocks);
    const long long b1 = min(b0 + share, (long long)p.num_blocks);
    const bool vectors = (reinterpret_cast<uintptr_t>(p.extra) & 15) == 0;
    auto gone_of = [&](long long b) {  // of blocks b .. b + kOwn - 1
        unsigned int gone = 0;
        if (b + kOwn <= b1 && vectors) {
            int4 x[kOwn / 4];
#pragma unroll
            for (int i = 0; i < kOwn / 4; ++i)
                x[i] = *reinterpret_cast<const int4 *>(p.extra + b + 4 * i);
#pragma unroll
            for (int i = 0; i < kOwn / 4; ++i)
                gone |= ((unsigned int)x[i].x >> 31 | (unsigned int)x[i].y >> 31 << 1 | (unsigned int)x[i].z >> 31 << 2 |
                         (unsigned int)x[i].w >> 31 << 3)
                        << (4 * i);
        } else {
            for (int i = 0; i < kOwn && b + i < b1; ++i)
                gone |= (p.extra[b + i] < 0 ? 1u : 0u) << i;
        }
        return gone;
    };
    const long long step = (long long)kEndThreads * kOwn;
    const unsigned int first_gone = gone_of(b0 + (long long)tid * kOwn);
    int mine = __popc(first_gone);
    for (long long b = b0 + tid * kOwn + step; b < b1; b += step)
        mine += __popc(gone_of(b));
    // the children that want a copy, kEndThreads of them a CTA at a time
    auto state_of = [&](int i) { return i < p.children ? p.granted[i] : (int)kEmpty; };
    int state = state_of(rank * kEndThreads + tid);
    if (tid == 0)
        freed = 0;
    wanted_here = 0;
    __syncthreads();
    mine = __reduce_add_sync(0xffffffffu, mine);
    if ((tid & 31) == 0 && mine)
        atomicAdd(&freed, mine);
    const unsigned int wants_mask = __ballot_sync(0xffffffffu, state == kWantsCopy);
    if ((tid & 31) == 0 && wants_mask)
        atomicAdd(&wanted_here, __popc(wants_mask));
    cluster.sync();
    long long before = 0, all = 0;
    int wanted = 0, round_wants = 0;  // wanted: by the children before this CTA's
    for (int r = 0; r < kEndCtas; ++r) {
        const int n = *cluster.map_shared_rank(&freed, r), w = *cluster.map_shared_rank(&wanted_here, r);
        before += r < rank ? n : 0;
        all += n;
        wanted += r < rank ? w : 0;
        round_wants += w;
    }
    if (freed > 0) {
        long long at = had + before;
        for (long long b = b0; b < b1; b += step) {
            const long long own = b + (long long)tid * kOwn;
            unsigned int gone = b == b0 ? first_gone : gone_of(own);
            int total;
            long long k = at + sum_before(__popc(gone), &total, part);
            while (gone) {
                const long long id = own + __ffs(gone) - 1;
                gone &= gone - 1;
                if (k < p.num_blocks)  // (past it: the list held blocks that were in use)
                    p.free_list[k] = (int)id;
                p.extra[id] = 0;
                ++k;
            }
            at += total;
        }
    }
    cluster.sync();  // the free list is whole, num_free and the counts have been read
    const int have = (int)min(had + all, (long long)p.num_blocks);

    // copies, in the children's order
    int total_wants = 0;
    for (int c = 0; c < p.children; c += kEndCtas * kEndThreads) {
        const int i = c + rank * kEndThreads + tid;
        if (c > 0) {  // (more than kEndCtas kEndThreads children: count the next ones)
            state = state_of(i);
            int total;
            sum_before(state == kWantsCopy ? 1 : 0, &total, part);
            cluster.sync();
            wanted_here = total;
            cluster.sync();
            wanted = total_wants;
            round_wants = 0;
            for (int r = 0; r < kEndCtas; ++r) {
                const int w = *cluster.map_shared_rank(&wanted_here, r);
                wanted += r < rank ? w : 0;
                round_wants += w;
            }
        }
        total_wants += round_wants;
        const bool wants = state == kWantsCopy;
        int total;
        const int k = wanted + sum_before(wants ? 1 : 0, &total, part);
        bool refused = false;
        if (i < p.children) {
            int len = 0, src = -1, dst = -1, says = state;
            if (state != kEmpty) {
                const int parent = p.parents[i];
                const Row row = row_of(p, parent);
                len = row.len;
                if (wants && k < have) {
                    const size_t last = (size_t)row.blocks - 1;
                    src = p.tables_in[(size_t)parent * p.max_blocks + last];
                    dst = p.free_list[have - 1 - k];
                    p.tables_out[(size_t)i * p.max_blocks + last] = dst;
                    says = kContinues;
                } else if (wants) {
                    len = 0;
                    says = kRefused;
                    refused = true;
                }
            }
            p.context_lens_out[i] = len;
            p.pairs[2 * (size_t)i] = src;
            p.pairs[2 * (size_t)i + 1] = dst;
            p.granted[i] = says;
        }
        // A refused child's row is empty and holds no references (its parent's first child holds the
        // same full blocks, so none of them is freed here).  A warp goes through its own.
        unsigned int left = __ballot_sync(0xffffffffu, refused);
        while (left) {
            const int child = (i & ~31) + __ffs(left) - 1;
            left &= left - 1;
            const int parent = p.parents[child];
            const Row row = row_of(p, parent);
            for (int j = tid & 31; j < row.blocks; j += 32) {
                if (j < row.blocks - 1)
                    add_refs(p, p.tables_in[(size_t)parent * p.max_blocks + j], -1);
                p.tables_out[(size_t)child * p.max_blocks + j] = -1;
            }
        }
    }
    if (rank == 0 && tid == 0)
        *p.num_free_out = max(have - total_wants, 0);
    cluster.sync();  // nobody's shared memory is read any more
}

}  // namespace

cudaError_t launch_fork_tables(const ForkParams &p, cudaStream_t stream)
{
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kEndCtas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    const int n = p.rows > p.children ? p.rows : p.children;
    if (n > 0) {
        cfg.gridDim = dim3((unsigned)n, (unsigned)((p.max_blocks + (long long)kRowEntries - 1) / kRowEntries));
        cfg.blockDim = dim3(kRowThreads);
        cfg.numAttrs = 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, fork_rows_kernel, p);
        if (e != cudaSuccess)
            return e;
    }
    cfg.gridDim = dim3(kEndCtas);
    cfg.blockDim = dim3(kEndThreads);
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fork_end_kernel, p);
}

}  // namespace pagedkv

using namespace pagedkv;

extern "C" pa_status pa_fork_tables(int32_t *block_tables_out, const int32_t *block_tables, int max_blocks_per_seq,
                                    int32_t *context_lens_out, const int32_t *context_lens, int num_rows,
                                    const int32_t *parents, int num_children, int32_t *extra_refs,
                                    int32_t *free_list, int num_blocks, int32_t *num_free_out,
                                    const int32_t *num_free, int block_size, int32_t *copy_pairs,
                                    int32_t *granted, void *stream)
{
    if (num_rows < 0 || num_children < 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 || block_size <= 0)
        return PA_ERR_INVALID;
    if (!extra_refs || !free_list || !num_free_out || !num_free)
        return PA_ERR_INVALID;
    if (num_rows > 0 && (!block_tables || !context_lens))
        return PA_ERR_INVALID;
    if (num_children > 0 && (!block_tables_out || !context_lens_out || !parents || !copy_pairs || !granted))
        return PA_ERR_INVALID;
    // a new row is written while others may still be read
    if (num_rows > 0 && num_children > 0 &&
        (block_tables_out == block_tables || context_lens_out == context_lens))
        return PA_ERR_INVALID;
    for (const void *ptr : {(const void *)block_tables_out, (const void *)block_tables,
                            (const void *)context_lens_out, (const void *)context_lens, (const void *)parents,
                            (const void *)extra_refs, (const void *)free_list, (const void *)num_free_out,
                            (const void *)num_free, (const void *)copy_pairs, (const void *)granted})
        if (!aligned(ptr, 4))
            return PA_ERR_INVALID;
    if ((long long)num_blocks * block_size >= (1ll << 31) ||
        (long long)max_blocks_per_seq * block_size >= (1ll << 31))
        return PA_ERR_INVALID;
    // (each row looks through the parents, and a grid has at most 65535 parts of a row)
    if (num_rows > kForkMaxRows || num_children > kForkMaxRows || max_blocks_per_seq > 65535 * kRowEntries ||
        num_blocks > kMaxCount)
        return PA_ERR_UNSUPPORTED;
    ForkParams p;
    p.tables_out = block_tables_out;
    p.tables_in = block_tables;
    p.context_lens_out = context_lens_out;
    p.context_lens = context_lens;
    p.parents = parents;
    p.extra = extra_refs;
    p.free_list = free_list;
    p.num_free_out = num_free_out;
    p.num_free = num_free;
    p.pairs = copy_pairs;
    p.granted = granted;
    p.max_blocks = max_blocks_per_seq;
    p.rows = num_rows;
    p.children = num_children;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    const cudaError_t e = launch_fork_tables(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : cuda_fail(e);
}
