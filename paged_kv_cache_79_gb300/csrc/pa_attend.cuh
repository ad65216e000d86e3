// Attention of several query tokens per sequence over the paged cache (pa_attend): the
// schedule that its kernels share, and their launchers.
//
// An item is (sequence, kv head, up to kSub heads of its group, a run of query tokens): the
// rows (token, head) of an item share every K and V row that they read.  Items are laid out in
// a stream, each with a cost of the keys that it sees plus a fixed charge, and the stream is cut
// into equal shares, one per CTA of a persistent grid: long sequences, causal tiles of every
// length and single query tokens all load every SM alike.  A cut inside an item falls on a
// tile of keys; the CTAs on both sides then leave partial rows (unnormalised output, maximum,
// sum in fp32), which a second kernel merges by the log-sum-exp rule.  A cut near an item's end
// moves to the end, so that few items pay for it.  The items' costs have closed forms, so a CTA
// finds its share from the lengths alone, without a pass over the items and without workspace
// that has to be cleared.
#pragma once

#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pagedkv {

constexpr int kAttendRows = 256;     // rows of an item at most
// An item's fixed cost, in keys: a tile of 128 takes 1.4 us, an item 2.4 to 3.8 us more.
constexpr int kAttendCharge = 320;
// A share's cost at least.  It is at least a tile of any item that can be cut (two tiles or more:
// charge + 2 * 128 <= 2 * 320), so two cuts of an item never fall on the same tile and every CTA
// between them has a part.
constexpr int kAttendMinShare = 320;
static_assert(kAttendCharge + 2 * 128 <= 2 * kAttendMinShare, "a part for every CTA");
constexpr int kF32TileRows = 64;     // rows of an item of the fp32 kernel

struct AttendItem {
    int s, u, j;         // sequence, (kv head, head chunk), run of query tokens
    int q0, n, T;        // the sequence's first query row, query tokens, keys
    int seen;            // keys that the item's last token sees
    int tiles;           // tiles of keys
    long long at;        // position of the item in the stream
    long long cost;
};

template <int kKeys>
struct AttendWalk {
    const AttendParams &p;
    AttendItem it;
    long long total, share_lo, share_hi;  // the stream, this CTA's share of it
    int snap;                             // a cut closer to an item's end (tiles) moves there
    int runs;                             // of the sequence

    __device__ __forceinline__ explicit AttendWalk(const AttendParams &params) : p(params) {}

    static __device__ __forceinline__ void sequence(const AttendParams &p, int s, int &q0, int &n, int &T)
    {
        const int a = min(max(p.query_start[s], 0), p.num_rows);
        const int b = min(max(p.query_start[s + 1], a), p.num_rows);
        q0 = a;
        n = b - a;
        T = (int)min((long long)max(p.context_lens[s], 0), (long long)p.max_blocks * p.block_size);
    }
    static __device__ __forceinline__ int runs_of(const AttendParams &p, int n)
    {
        return (n + p.tokens_per_item - 1) / p.tokens_per_item;
    }
    // Keys that the last token of run j sees.
    static __device__ __forceinline__ int seen_by(const AttendParams &p, int n, int T, int j)
    {
        if (!p.causal)
            return T;
        const long long last = min((long long)n, (long long)(j + 1) * p.tokens_per_item);
        return (int)max((long long)T - n + last, 0ll);
    }
    // Cost of run j, which sees `seen` keys; one of few tokens goes through its keys twice as fast.
    static __device__ __forceinline__ long long cost_of(const AttendParams &p, int n, int j, int seen)
    {
        const bool few = n - (long long)j * p.tokens_per_item <= p.few_tokens;
        return kAttendCharge + (few ? ((long long)seen + 1) / 2 : (long long)seen);
    }
    // Cost of runs 0 .. j - 1 of one unit of the sequence.  (All but the last are whole.)
    static __device__ __forceinline__ long long before(const AttendParams &p, int n, int T, int j)
    {
        const long long t = p.tokens_per_item;
        const bool all = j > 0 && (long long)j * t >= n;  // the last run is among them
        const int full = all ? j - 1 : j;
        long long sum = (long long)full * kAttendCharge + (all ? cost_of(p, n, j - 1, T) : 0);
        if (!p.causal)
            return sum + (long long)full * T;
        const long long over = (long long)T - n;
        const long long i0 = over >= 0 ? 0 : min(-over / t, (long long)full);
        const long long m = full - i0;
        return sum + m * over + t * ((i0 + 1 + full) * m / 2);
    }

    __device__ __forceinline__ void set(int s, int u, int j, int q0, int n, int T, long long at)
    {
        it.s = s;
        it.u = u;
        it.j = j;
        it.q0 = q0;
        it.n = n;
        it.T = T;
        it.at = at;
        it.seen = seen_by(p, n, T, j);
        it.tiles = (int)(((unsigned int)it.seen + (kKeys - 1)) / kKeys);  // (seen may be next to 2^31)
        it.cost = cost_of(p, n, j, it.seen);
    }
    // The next item of the stream; false behind the last.
    __device__ __forceinline__ bool next()
    {
        const long long at = it.at + it.cost;
        if (it.j + 1 < runs) {
            set(it.s, it.u, it.j + 1, it.q0, it.n, it.T, at);
            return true;
        }
        if (it.u + 1 < p.units) {
            set(it.s, it.u + 1, 0, it.q0, it.n, it.T, at);
            return true;
        }
        int s = it.s, q0, n, T;
        do {
            if (++s >= p.num_seqs)
                return false;
            sequence(p, s, q0, n, T);
        } while (n == 0);
        runs = runs_of(p, n);
        set(s, 0, 0, q0, n, T, at);
        return true;
    }
    // First tile of the item at or behind stream position x.
    __device__ __forceinline__ int cut(long long x) const
    {
        if (x <= it.at)
            return 0;
        if (x >= it.at + it.cost)
            return it.tiles;
        const int c = (int)((x - it.at) * it.tiles / it.cost);
        return c < snap ? 0 : it.tiles - c < snap ? it.tiles : c;
    }
    // The part of the item that is this CTA's: tiles [a, b); false: none.
    __device__ __forceinline__ bool part(int &a, int &b) const
    {
        a = cut(share_lo);
        b = cut(share_hi);
        return b > a || (it.tiles == 0 && it.at >= share_lo && it.at < share_hi);
    }
    __device__ __forceinline__ bool inside() const { return it.at < share_hi; }

    // Where CTA `cta`'s share of the stream begins; `ctas`: how many share it.
    __device__ __forceinline__ static long long start_of(long long total, int cta, int ctas)
    {
        return total / ctas * cta + total % ctas * cta / ctas;
    }

    // Finds the CTA's share and its first item (all threads of the CTA, kThreads of them;
    // scratch: shared memory).  False: the share is empty.
    template <int kThreads>
    __device__ __forceinline__ bool begin(long long (&scratch)[kThreads / 32 + 4])
    {
        constexpr int kWarps = kThreads / 32;
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        auto cost_of = [&](int s) -> long long {
            if (s >= p.num_seqs)
                return 0;
            int q0, n, T;
            sequence(p, s, q0, n, T);
            return n > 0 ? before(p, n, T, runs_of(p, n)) * p.units : 0;
        };
        // inclusive sum over the CTA's threads; *sum: all of them
        auto scan = [&](long long x, long long &sum) -> long long {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o)
                    x += y;
            }
            __syncthreads();
            if (lane == 31)
                scratch[warp] = x;
            __syncthreads();
            long long add = 0;
            sum = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                add += w < warp ? scratch[w] : 0;
                sum += scratch[w];
            }
            return x + add;
        };
        total = 0;
        long long first = 0, mine = 0;  // of the first kThreads sequences
        for (int s0 = 0; s0 < p.num_seqs; s0 += kThreads) {
            long long sum;
            const long long c = cost_of(s0 + tid), in = scan(c, sum);
            if (s0 == 0) {
                first = in;
                mine = c;
            }
            total += sum;
        }
        const int ctas = (int)max(1ll, min((long long)gridDim.x, total / kAttendMinShare));
        const int cta = blockIdx.x;
        share_lo = cta < ctas ? start_of(total, cta, ctas) : total;
        share_hi = cta < ctas ? start_of(total, cta + 1, ctas) : total;
        snap = max(1, (int)min(total / ctas / (16 * kKeys), 1ll << 20));
        if (share_lo >= share_hi) {
            if (tid == 0)
                p.cuts[cta] = AttendCut{};
            return false;
        }
        // the sequence that holds share_lo
        long long base = 0;
        for (int s0 = 0; s0 < p.num_seqs; s0 += kThreads) {
            long long sum = 0, in = first, c = mine;
            if (p.num_seqs > kThreads) {
                c = cost_of(s0 + tid);
                in = scan(c, sum);
            }
            if (base + in > share_lo && base + in - c <= share_lo) {
                scratch[kWarps] = s0 + tid;
                scratch[kWarps + 1] = base + in - c;
            }
            base += sum;
        }
        __syncthreads();
        const int s = (int)scratch[kWarps];
        const long long at = scratch[kWarps + 1];
        int q0, n, T;
        sequence(p, s, q0, n, T);
        runs = runs_of(p, n);
        const long long unit = before(p, n, T, runs);
        const int u = (int)((share_lo - at) / unit);
        const long long r = share_lo - at - u * unit;
        int lo = 0, hi = runs - 1;  // the last run that begins at or before r
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (before(p, n, T, mid) <= r)
                lo = mid;
            else
                hi = mid - 1;
        }
        set(s, u, lo, q0, n, T, at + u * unit + before(p, n, T, lo));
        // one thread leaves what the merge needs
        if (tid == 0) {
            AttendCut cutinfo = {};
            const int a = cut(share_lo);
            if (a > 0 && a < it.tiles && cut(start_of(total, cta - 1, ctas)) == 0) {
                int last = cta;
                while (last + 1 < ctas && cut(start_of(total, last + 1, ctas)) < it.tiles)
                    ++last;
                const AttendRows rows = rows_of(p, it);
                cutinfo.parts = last - cta + 2;
                cutinfo.token0 = rows.token0;
                cutinfo.tokens = rows.tokens;
                cutinfo.head0 = rows.head0;
                cutinfo.heads = rows.heads;
            }
            p.cuts[cta] = cutinfo;
        }
        return true;
    }

    struct AttendRows {
        int token0, tokens, head0, heads, kv;
    };
    static __device__ __forceinline__ AttendRows rows_of(const AttendParams &p, const AttendItem &it)
    {
        AttendRows r;
        const int first = it.j * p.tokens_per_item;
        r.token0 = it.q0 + first;
        r.tokens = min(it.n - first, p.tokens_per_item);
        r.kv = it.u / p.head_chunks;
        const int h = (it.u - r.kv * p.head_chunks) * p.heads_per_item;
        r.head0 = r.kv * p.group + h;
        r.heads = min(p.group - h, p.heads_per_item);
        return r;
    }
};

// Exponents (log2) that a row's base lies below the maximum that it was taken from.
template <typename T>
constexpr float kAttendBelow = std::is_same<T, __half>::value ? 11.0f : 0.0f;

// A row's log sum exp from its base m (log2 units) and its sum l over exp2(score - m).  (The
// base's distance is taken out of both first, so that neither is rounded at a larger size.)
template <typename T>
__device__ __forceinline__ float attend_lse(float m, float l)
{
    constexpr float kBelow = kAttendBelow<T>;
    const float scale = kBelow == 0.f ? 1.f : 1.f / (float)(1 << (int)kBelow);
    return l == 0.f ? -INFINITY : ((m + kBelow) + log2f(l * scale)) * 0.6931471805599453f;
}

// Partial rows of CTA c: slot 0 holds the item that its start cuts, slot 1 an item that
// begins in its share and is cut by its end; kAttendRows rows each, or fewer (max_rows).
__device__ __forceinline__ size_t attend_part_row(const AttendParams &p, int cta, int slot)
{
    return ((size_t)cta * 2 + slot) * p.part_rows;
}

cudaError_t launch_attend_f32(const AttendLaunch &L, cudaStream_t stream);
cudaError_t launch_attend_f16(const AttendLaunch &L, cudaStream_t stream);
cudaError_t launch_attend_bf16(const AttendLaunch &L, cudaStream_t stream);
cudaError_t launch_attend_merge(const AttendLaunch &L, int dtype, cudaStream_t stream);

}  // namespace pagedkv
