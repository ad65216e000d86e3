// Block tables and slot maps built on the GPU from request lengths: one step of the
// block allocator (CSDN tutorial "PagedAttention实战" §2.2 BlockManager, §3.1 append_kv)
// for a batch whose blocks are not shared, without the host.
//
// Request i has len_i tokens in ceil(len_i / B) blocks.  Requests with new_i < 0 give
// their blocks back, in request and table order, to the end of the free list; then the
// others take new_i tokens each, popping blocks from the end in request order.  Which
// request gets which entry follows from prefix sums over the requests, so all of it runs
// in one launch: each CTA of a cluster scans the requests, 1024 at a time, and the
// cluster's threads share the rows of the slot map and the new table entries, finding
// each one's request by binary search in the scanned sums.
//
// Bound by latency: a decode step's few kilobytes take two scans and two dependent reads
// of the free list or the table.  A cluster, not a grid, because the free list's new
// entries must be seen by every CTA, and the lengths read by all before one CTA
// overwrites them, which a cluster barrier gives without a second launch.  A long slot
// map (prompts) is written by a second kernel over the whole GPU, from the tables and
// lengths that the first has made.  256 requests with a token each take 5.1 us back to back,
// 64 prompts of up to 8000 tokens 10.4 (49 with the cluster writing the slot map), 1001
// mixed requests 11.8 (16.3).
#include <cooperative_groups.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pagedkv {

namespace {

constexpr int kTabThreads = 1024;
// CTAs of the cluster: one alone is never faster, and 1071 requests that release 100 of
// 4000 tokens take 25.0 us with one, 17.2 with four, 15.6 with eight.
constexpr int kTabCtas = 8;
// Up to this many slots the cluster writes the slot map too; above, build_slots_kernel.
// One kernel against two, us: 1 request, 512 slots 4.9 / 6.5, 4096 5.1 / 6.5, 8192 5.3 / 6.8,
// 16384 6.6 / 7.2, 65536 13.4 / 7.3; 1000 requests, 4000 slots 6.0 / 8.3, 8000 6.0 / 8.3, 16000
// 7.7 / 8.8, 65000 15.3 / 8.4.
constexpr int kTabFew = 4096;

// Inclusive sums of a and b over the CTA's threads; totals in ta, tb.
__device__ __forceinline__ void scan2(long long &a, long long &b, long long &ta, long long &tb,
                                      long long (&part)[2][32])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
            a += x;
            b += y;
        }
    }
    __syncthreads();  // the previous scan's sums have been read
    if (lane == 31) {
        part[0][warp] = a;
        part[1][warp] = b;
    }
    __syncthreads();
    long long x = part[0][lane], y = part[1][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) {
            x += u;
            y += v;
        }
    }
    ta = __shfl_sync(0xffffffffu, x, 31);
    tb = __shfl_sync(0xffffffffu, y, 31);
    if (warp > 0) {
        a += __shfl_sync(0xffffffffu, x, warp - 1);
        b += __shfl_sync(0xffffffffu, y, warp - 1);
    }
}

// First thread whose inclusive sum passes x.
__device__ __forceinline__ int owner(const long long *incl, long long x)
{
    int lo = 0, hi = kTabThreads - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (incl[mid] > x)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

// Blocks of B tokens that hold `tokens`, both below 2^31 (their sum may pass that).
__device__ __forceinline__ int blocks_of(long long tokens, int B)
{
    return (int)(((unsigned int)tokens + (unsigned int)(B - 1)) / (unsigned int)B);
}

__global__ void __launch_bounds__(kTabThreads) build_tables_kernel(const __grid_constant__ TablesParams p)
{
    namespace cg = cooperative_groups;
    __shared__ long long part[2][32];
    __shared__ long long tok_incl[kTabThreads], blk_incl[kTabThreads];
    __shared__ int s_len[kTabThreads];
    cg::cluster_group cluster = cg::this_cluster();
    dev::grid_dependency_wait();
    dev::grid_launch_dependents();
    const int tid = threadIdx.x;
    const long long first = (long long)cluster.block_rank() * kTabThreads + tid;
    const long long stride = (long long)cluster.num_blocks() * kTabThreads;
    const bool writer = cluster.block_rank() == 0;
    const int B = p.block_size, W = p.max_blocks;
    const long long cap = (long long)W * B;

    // released requests' blocks go to the end of the free list
    const long long had = min(max(*p.num_free, 0), p.num_blocks);
    long long have = had;
    int len = 0, want = 0;
    for (int s0 = 0; s0 < p.num_seqs; s0 += kTabThreads) {
        const int s = s0 + tid;
        len = s < p.num_seqs ? max(p.context_lens[s], 0) : 0;
        want = s < p.num_seqs ? p.new_tokens[s] : 0;
        if (!__syncthreads_or(want < 0))
            continue;
        long long gone = want < 0 ? blocks_of(min((long long)len, cap), B) : 0, none = 0, total, zero;
        scan2(gone, none, total, zero, part);
        blk_incl[tid] = gone;
        __syncthreads();
        for (long long i = first; i < total; i += stride) {
            const int o = owner(blk_incl, i);
            const long long j = i - (o > 0 ? blk_incl[o - 1] : 0);
            // (a request released twice over could pass the list's end)
            if (have + i < p.num_blocks)
                p.free_list[have + i] = p.block_tables[(size_t)(s0 + o) * W + j];
        }
        __syncthreads();
        have = min(have + total, (long long)p.num_blocks);
    }
    cluster.sync();  // every CTA has read the lengths and sees the whole free list

    long long need_before = 0, want_before = 0, tok_before = 0, blk_before = 0;
    for (int s0 = 0; s0 < p.num_seqs; s0 += kTabThreads) {
        const int s = s0 + tid;
        if (p.num_seqs > kTabThreads) {
            len = s < p.num_seqs ? max(p.context_lens[s], 0) : 0;
            want = s < p.num_seqs ? p.new_tokens[s] : 0;
            cluster.sync();  // read by every CTA before the writer goes on
        }
        const int nb = blocks_of(min((long long)len, cap), B);
        const bool fits = want <= 0 || (long long)len + want <= cap;
        const int n = fits && want > 0 ? want : 0;
        const int need = n > 0 ? blocks_of((long long)len + n, B) - nb : 0;
        long long ni = need, wi = n, nt, wt;
        scan2(ni, wi, nt, wt, part);
        const bool ok = want <= 0 || (fits && (need == 0 || need_before + ni <= have) &&
                                      want_before + wi <= p.num_slots);
        need_before += nt;
        want_before += wt;
        // sums over the granted requests: those over all where none is refused
        long long ti = wi, bi = ni, tt = wt, bt = nt;
        const int got = ok ? n : 0;
        if (__syncthreads_or(!ok)) {
            ti = got;
            bi = ok ? need : 0;
            scan2(ti, bi, tt, bt, part);
        }
        tok_incl[tid] = ti;
        blk_incl[tid] = bi;
        s_len[tid] = len;
        __syncthreads();
        if (writer && s < p.num_seqs) {
            p.context_lens_out[s] = want < 0 ? 0 : len + got;
            p.granted[s] = ok ? got : -1;
            p.query_start[s + 1] = (int)(tok_before + ti);
        }
        // entry of the free list that new block i of request o gets
        auto popped = [&](int o, long long i) {
            const long long at = have - 1 - (blk_before + (o > 0 ? blk_incl[o - 1] : 0) + i);
            return at >= 0 && at < p.num_blocks ? p.free_list[at] : -1;
        };
        for (long long i = first; i < bt; i += stride) {
            const int o = owner(blk_incl, i);
            const long long k = i - (o > 0 ? blk_incl[o - 1] : 0);
            const int nb_o = blocks_of(s_len[o], B);
            p.block_tables[(size_t)(s0 + o) * W + nb_o + k] = popped(o, k);
        }
        for (long long i = first; i < tt && !p.slots_apart; i += stride) {
            const int o = owner(tok_incl, i);
            const int pos = s_len[o] + (int)(i - (o > 0 ? tok_incl[o - 1] : 0));
            const int j = pos / B, nb_o = blocks_of(s_len[o], B);
            const int id = j < nb_o ? p.block_tables[(size_t)(s0 + o) * W + j] : popped(o, j - nb_o);
            p.slots[tok_before + i] = id >= 0 ? (int64_t)id * B + pos % B : -1;
        }
        tok_before += tt;
        blk_before += bt;
        __syncthreads();  // the sums are read before the next chunk's take their place
    }
    for (long long i = tok_before + first; i < p.num_slots && !p.slots_apart; i += stride)
        p.slots[i] = -1;
    if (writer && tid == 0) {
        p.query_start[0] = 0;
        *p.num_free_out = (int)(have - blk_before);
    }
}

// The slot map from the finished tables: kSlotsPerWarp consecutive slots per warp, whose
// requests one search finds (few, since a warp's reads of them depend on each other: 64
// prompts of up to 8000 tokens take 10.5 us, with 256 11.9; 1001 mixed requests 11.8 and
// 16.1; with 32 slots 10.9 and 11.0).
constexpr int kSlotWarps = 8;
constexpr int kSlotsPerWarp = 64;
__global__ void __launch_bounds__(32 * kSlotWarps) build_slots_kernel(const __grid_constant__ TablesParams p)
{
    dev::grid_dependency_wait();
    dev::grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long base = ((long long)blockIdx.x * kSlotWarps + (threadIdx.x >> 5)) * kSlotsPerWarp;
    const int total = p.query_start[p.num_seqs];
    const int B = p.block_size;
    int s = -1, end = 0;  // the lane's request, and the end of its slots
    for (int k = 0; k < kSlotsPerWarp / 32; ++k) {
        const long long t0 = base + k * 32;
        if (t0 >= p.num_slots)
            return;
        const int t = (int)t0 + lane;
        if (t0 < total && !__all_sync(0xffffffffu, s >= 0 && t < end)) {
            s = min(dev::find_sequence(p.query_start, p.num_seqs, (int)t0, lane,
                                       k == 0 ? -1 : __shfl_sync(0xffffffffu, s, 31)), p.num_seqs - 1);
            end = p.query_start[s + 1];
        }
        int64_t slot = -1;
        if (t < total) {
            const int pos = p.context_lens_out[s] - (end - t);
            const int id = p.block_tables[(size_t)s * p.max_blocks + pos / B];
            slot = id >= 0 ? (int64_t)id * B + pos % B : -1;
        }
        if (t < p.num_slots)
            p.slots[t] = slot;
    }
}

}  // namespace

cudaError_t launch_build_tables(TablesParams p, cudaStream_t stream)
{
    p.slots_apart = p.num_slots > kTabFew && p.num_seqs > 0;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kTabCtas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kTabCtas);
    cfg.blockDim = dim3(kTabThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, build_tables_kernel, p);
    if (e != cudaSuccess || !p.slots_apart)
        return e;
    const int per_cta = kSlotWarps * kSlotsPerWarp;
    cfg.gridDim = dim3((unsigned)((p.num_slots + (long long)per_cta - 1) / per_cta));
    cfg.blockDim = dim3(32 * kSlotWarps);
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, build_slots_kernel, p);
}

}  // namespace pagedkv
