// fa_pages_kernel.cuh -- page tables and slot maps of a step from the sequences'
// lengths, and pages given back, on sm_103a.
//
// need(b) = pages(len + n) - pages(len); prefix sums of n place a sequence's rows, those of
// need its pages in the ring.  What bounds it is no traffic (8 bytes a row) but a chain:
// lengths, two sums over the batch, then per row a search for its sequence, its page, its
// slot.  So one launch of one cluster does all: every block takes the sums over the whole
// batch by itself (a few words a thread), which costs less than a second launch, and the
// rows and pages are shared out among the blocks.  The searches run in shared memory.
#pragma once

#include "fa_common.cuh"

namespace fa {
namespace pages {

constexpr int kThreads = 512;
constexpr int kBlocks = 8;  // one cluster
constexpr int kMaxBatch = 16384;
constexpr int kRows = 4;    // neighbouring rows a thread

// Dynamic shared memory: [B + 1] first rows, [B] pages up to and with a sequence.
inline __host__ __device__ size_t smem_bytes(int B) { return static_cast<size_t>(2 * B + 1) * 4; }

struct Pool {
    int *ring;
    int size;
    const long long *counts;
    long long *out;
};
struct Lengths {
    const int *had, *other;  // tokens; new ones, or those to keep
    int B, log2_page;
};

__device__ __forceinline__ void cluster_meet()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// Inclusive sum over the block's threads of x, and the block's total.
__device__ __forceinline__ long long block_scan(long long x, long long *warps, long long &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o)
            x += y;
    }
    __syncthreads();  // earlier reads of warps are done
    if (lane == 31)
        warps[warp] = x;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp)
            x += warps[w];
        total += warps[w];
    }
    return x;
}

// First i of [0, n) with a[i] > x; n if there is none.
__device__ __forceinline__ int first_above(const int *a, int n, int x)
{
    int lo = 0;
    while (n > 0) {
        const int half = n >> 1;
        if (a[lo + half] > x) {
            n = half;
        } else {
            lo += half + 1;
            n -= half + 1;
        }
    }
    return lo;
}

__device__ __forceinline__ int up_to(long long x) { return x < 0x7fffffff ? static_cast<int>(x) : 0x7fffffff; }
__device__ __forceinline__ long long pages_of(long long tokens, int log2_page)
{
    return (tokens + (1 << log2_page) - 1) >> log2_page;
}

// Free pages, and where in the ring the x-th of them lies.
struct Ring {
    int size;
    unsigned begin, end;  // places of the first page and of the first behind the last
    int free;
    bool bad;
    __device__ explicit Ring(const Pool &p) : size(p.size)
    {
        const long long taken = p.counts[0], given = p.counts[1];
        bad = taken < 0 || given < taken || given - taken > p.size;
        free = bad ? 0 : static_cast<int>(given - taken);
        begin = bad ? 0 : static_cast<unsigned>(taken % p.size);
        end = bad ? 0 : static_cast<unsigned>(given % p.size);
    }
    // x < size
    __device__ int place(unsigned from, int x) const
    {
        const unsigned at = from + static_cast<unsigned>(x);
        return static_cast<int>(at < static_cast<unsigned>(size) ? at : at - size);
    }
};

__global__ void __cluster_dims__(kBlocks, 1, 1) __launch_bounds__(kThreads)
    fa_cache_plan_kernel(Pool pool, Lengths in, int *__restrict__ table, long long table_stride, int max_pages,
                         int *__restrict__ cu_seqlens, int *__restrict__ ends, int *__restrict__ positions,
                         int *__restrict__ slots, int T, unsigned int *status)
{
    extern __shared__ int smem[];
    __shared__ long long warps[kThreads / 32];
    __shared__ int taken_all;
    int *cu = smem, *until = smem + in.B + 1;
    const int t = threadIdx.x, wide = kThreads * kBlocks;
    const int mine = blockIdx.x * kThreads + t;
    const Ring ring(pool);
    const int log2_page = in.log2_page;
    const long long cap = static_cast<long long>(max_pages) << log2_page;
    bool bad = ring.bad && mine == 0;
    if (t == 0)
        taken_all = 0;
    // this thread's sequences, one after the other
    const int each = (in.B + kThreads - 1) / kThreads;
    const int b0 = min(in.B, t * each), b1 = min(in.B, b0 + each);
    long long rows = 0, total;
    for (int b = b0; b < b1; ++b)
        rows += max(0, in.had[b] < 0 ? 0 : in.other[b]);
    const long long first_row = block_scan(rows, warps, total) - rows;
    const int all_rows = up_to(total);
    long long row = first_row, need = 0;
    auto needs = [&](int b, long long begin, int &n) -> long long {  // -1: it does not fit
        const long long had = in.had[b];
        n = had < 0 ? 0 : max(0, in.other[b]);
        if (had < 0 || in.other[b] < 0 || had + n > cap || begin + n > T)
            return -1;
        return pages_of(had + n, log2_page) - pages_of(had, log2_page);
    };
    for (int b = b0; b < b1; ++b) {
        int n;
        need += max(0ll, needs(b, row, n));
        row += n;
    }
    long long pages = block_scan(need, warps, total) - need;
    row = first_row;
    for (int b = b0; b < b1; ++b) {
        int n;
        const long long more = needs(b, row, n);
        pages += max(0ll, more);
        const bool served = more == 0 || (more > 0 && pages <= ring.free);
        cu[b] = up_to(row);
        until[b] = up_to(pages);
        if (served && more > 0)
            atomicMax(&taken_all, until[b]);
        if (b / each % kBlocks == blockIdx.x) {  // its outputs are this block's to write
            cu_seqlens[b] = up_to(row);
            ends[b] = served ? in.had[b] + n : in.had[b];
            bad |= more < 0;
        }
        row += n;
    }
    if (t == 0)
        cu[in.B] = all_rows;
    if (mine == 0) {
        cu_seqlens[in.B] = all_rows;
        bad |= total > 0x7fffffff;
    }
    __syncthreads();
    const int taken = taken_all;
    // the pages taken: those of refused sequences come behind them
    for (int j = mine; j < taken; j += wide) {
        const int b = first_above(until, in.B, j);
        const int before = b > 0 ? until[b - 1] : 0;
        const long long at = pages_of(in.had[b], log2_page) + (j - before);
        table[b * table_stride + at] = pool.ring[ring.place(ring.begin, j)];
    }
    // the rows
    for (long long t0 = static_cast<long long>(mine) * kRows; t0 < T; t0 += static_cast<long long>(wide) * kRows) {
        int b = t0 < all_rows ? first_above(cu + 1, in.B, static_cast<int>(t0)) : in.B;
        int p[kRows], s[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int at = static_cast<int>(t0) + u;  // behind T it is written nowhere
            p[u] = s[u] = -1;
            while (b < in.B && at >= cu[b + 1])
                ++b;
            if (b >= in.B || t0 + u >= T)
                continue;
            const long long had = in.had[b];
            const int before = b > 0 ? until[b - 1] : 0;
            const int n = cu[b + 1] - cu[b];
            // a row has a sequence with n > 0: it was refused if it did not fit, or its pages did not
            if (had + n > cap || cu[b + 1] > T || (until[b] > before && until[b] > ring.free))
                continue;
            const int pos = static_cast<int>(had) + at - cu[b];
            const long long column = pos >> log2_page, old = pages_of(had, log2_page);
            const int page = column < old ? table[b * table_stride + column]
                                          : pool.ring[ring.place(ring.begin, before + static_cast<int>(column - old))];
            p[u] = pos;
            if (page >= 0 && page < pool.size)
                s[u] = (page << log2_page) + (pos & ((1 << log2_page) - 1));
            else
                bad = true;
        }
        if (t0 + kRows <= T && ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(slots)) & 15) == 0) {
            *reinterpret_cast<int4 *>(positions + t0) = make_int4(p[0], p[1], p[2], p[3]);
            *reinterpret_cast<int4 *>(slots + t0) = make_int4(s[0], s[1], s[2], s[3]);
        } else {
#pragma unroll
            for (int u = 0; u < kRows; ++u)
                if (t0 + u < T) {
                    positions[t0 + u] = p[u];
                    slots[t0 + u] = s[u];
                }
        }
    }
    if (bad)
        atomicOr(status, kStatusBounds);
    const long long counts0 = pool.counts[0], counts1 = pool.counts[1];
    cluster_meet();  // every block has read the counts, which may be the ones that are written
    if (mine == 0) {
        pool.out[0] = counts0 + taken;
        pool.out[1] = counts1;
    }
}

__global__ void __cluster_dims__(kBlocks, 1, 1) __launch_bounds__(kThreads)
    fa_cache_trim_kernel(Pool pool, Lengths in, const int *__restrict__ table, long long table_stride, int max_pages,
                         unsigned int *status)
{
    extern __shared__ int smem[];
    __shared__ long long warps[kThreads / 32];
    __shared__ int back_all;
    int *until = smem;
    const int t = threadIdx.x, wide = kThreads * kBlocks;
    const int mine = blockIdx.x * kThreads + t;
    const Ring ring(pool);
    const int log2_page = in.log2_page;
    const long long cap = static_cast<long long>(max_pages) << log2_page;
    const int room = ring.bad ? 0 : ring.size - ring.free;
    bool bad = ring.bad && mine == 0;
    if (t == 0)
        back_all = 0;
    const int each = (in.B + kThreads - 1) / kThreads;
    const int b0 = min(in.B, t * each), b1 = min(in.B, b0 + each);
    auto gives = [&](int b) -> long long {  // -1: lengths that are none
        const int had = in.had[b], keep = in.other[b];
        return keep < 0 || keep > had || had > cap ? -1 : pages_of(had, log2_page) - pages_of(keep, log2_page);
    };
    long long sum = 0, total;
    for (int b = b0; b < b1; ++b)
        sum += max(0ll, gives(b));
    long long pages = block_scan(sum, warps, total) - sum;
    for (int b = b0; b < b1; ++b) {
        const long long n = gives(b);
        pages += max(0ll, n);
        until[b] = up_to(pages);
        if (n > 0 && pages <= room)
            atomicMax(&back_all, until[b]);
        if (mine == t)
            bad |= n < 0 || (n > 0 && pages > room);
    }
    __syncthreads();
    const int back = back_all;
    for (int j = mine; j < back; j += wide) {
        const int b = first_above(until, in.B, j);
        const int before = b > 0 ? until[b - 1] : 0;
        const int page = table[b * table_stride + pages_of(in.other[b], log2_page) + (j - before)];
        bad |= page < 0 || page >= pool.size;
        pool.ring[ring.place(ring.end, j)] = page;
    }
    if (bad)
        atomicOr(status, kStatusBounds);
    const long long counts0 = pool.counts[0], counts1 = pool.counts[1];
    cluster_meet();  // every block has read the counts, which may be the ones that are written
    if (mine == 0) {
        pool.out[0] = counts0;
        pool.out[1] = counts1 + back;
    }
}

}  // namespace pages
}  // namespace fa
