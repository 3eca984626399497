// fa_pages_kernel.cuh -- page tables and slot maps of a step from the sequences'
// lengths, and pages given back, on sm_103a.
//
// need(b) = pages(len + n) - pages(len); prefix sums of n place a sequence's rows, those of
// need its pages in the ring.  What bounds it is no traffic (8 bytes a row) but a chain:
// lengths, two sums over the batch, then per row a search for its sequence, its page, its
// slot.  So one block does all of a step: sums over the batch, pages and, of up to kOwnRows
// rows, positions and slots, by searches in shared memory.  More rows (prompts) go to a
// second launch, which reads what the first has written.  On the GPU 256 sequences of 4
// tokens take 4.2 us, and as much to give some back; 64 with 130,000 new tokens 8.3 (one
// cluster of eight blocks for all of it took 22.8, the rows bound by those eight SMs).
#pragma once

#include "fa_cache_kernel.cuh"

namespace fa {
namespace pages {

constexpr int kThreads = 1024;
constexpr int kMaxBatch = 16384;
constexpr int kRows = 4;       // neighbouring rows a thread
constexpr int kOwnRows = 4096;  // that the first launch takes
constexpr int kRowThreads = 256;

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
struct Rows {
    int *positions, *slots;
    int T;

    // Rows t0 .. t0 + kRows - 1 at once where they lie so.
    __device__ void write(long long t0, const int (&p)[kRows], const int (&s)[kRows]) const
    {
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
};

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
    // every warp sums the warps' totals by itself
    long long y = warps[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o)
            y += z;
    }
    total = __shfl_sync(0xffffffffu, y, 31);
    const long long before = __shfl_sync(0xffffffffu, y, (warp + 31) & 31);
    return warp ? x + before : x;
}
static_assert(kThreads == 1024, "a warp has a lane for each warp's total");

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

// Free pages, and where in the ring the x-th of them lies.  One thread divides.
struct Ring {
    unsigned begin, end;  // places of the first page and of the first behind the last
    int free, bad;
    __device__ void read(const Pool &p)
    {
        const long long taken = p.counts[0], given = p.counts[1];
        bad = taken < 0 || given < taken || given - taken > p.size;
        free = bad ? 0 : static_cast<int>(given - taken);
        begin = bad ? 0 : static_cast<unsigned>(taken % p.size);
        end = begin + static_cast<unsigned>(free);
        end = end < static_cast<unsigned>(p.size) ? end : end - p.size;
    }
};
// x < size
__device__ __forceinline__ int place(int size, unsigned from, int x)
{
    const unsigned at = from + static_cast<unsigned>(x);
    return static_cast<int>(at < static_cast<unsigned>(size) ? at : at - size);
}

__global__ void __launch_bounds__(kThreads)
    fa_cache_plan_kernel(Pool pool, Lengths in, int *table, long long table_stride, int max_pages, int *cu_seqlens, int *ends,
                         Rows rows, unsigned int *status)
{
    extern __shared__ int smem[];
    __shared__ long long warps[kThreads / 32];
    __shared__ Ring ring;
    __shared__ int taken_all;
    int *cu = smem, *until = smem + in.B + 1;
    const int t = threadIdx.x;
    const int log2_page = in.log2_page;
    const long long cap = static_cast<long long>(max_pages) << log2_page;
    cache::wait_ahead();
    cache::let_next();
    if (t == kThreads - 1) {  // a thread that has no sequence in a batch of fewer
        ring.read(pool);
        taken_all = 0;
    }
    // this thread's sequences, one after the other
    const int each = (in.B + kThreads - 1) / kThreads;
    const int b0 = min(in.B, t * each), b1 = min(in.B, b0 + each);
    long long count = 0, total;
    for (int b = b0; b < b1; ++b)
        count += in.had[b] < 0 ? 0 : max(0, in.other[b]);
    const long long first_row = block_scan(count, warps, total) - count;
    const int all_rows = up_to(total);
    bool bad = t == 0 && (ring.bad || total > 0x7fffffff);
    long long row = first_row, need = 0;
    auto needs = [&](int b, long long begin, int &n) -> long long {  // -1: it does not fit
        const long long had = in.had[b];
        n = had < 0 ? 0 : max(0, in.other[b]);
        if (had < 0 || in.other[b] < 0 || had + n > cap || begin + n > rows.T)
            return -1;
        return pages_of(had + n, log2_page) - pages_of(had, log2_page);
    };
    for (int b = b0; b < b1; ++b) {
        int n;
        need += max(0ll, needs(b, row, n));
        row += n;
    }
    const long long first_page = block_scan(need, warps, total) - need;
    long long pages = first_page;
    row = first_row;
    for (int b = b0; b < b1; ++b) {
        int n;
        const long long more = needs(b, row, n);
        pages += max(0ll, more);
        const bool served = more == 0 || (more > 0 && pages <= ring.free);
        cu[b] = cu_seqlens[b] = up_to(row);
        until[b] = up_to(pages);
        if (served && more > 0)
            atomicMax(&taken_all, until[b]);
        ends[b] = served ? in.had[b] + n : in.had[b];
        bad |= more < 0;
        row += n;
    }
    if (t == 0)
        cu[in.B] = cu_seqlens[in.B] = all_rows;
    __syncthreads();
    const int taken = taken_all;
    // the pages taken: those of refused sequences come behind them; the last threads begin with them,
    // the first ones with the rows
    for (int j = kThreads - 1 - t; j < taken; j += kThreads) {
        const int b = first_above(until, in.B, j);
        const int before = b > 0 ? until[b - 1] : 0;
        const long long at = pages_of(in.had[b], log2_page) + (j - before);
        table[b * table_stride + at] = pool.ring[place(pool.size, ring.begin, j)];
    }
    const int own = rows.T <= kOwnRows ? rows.T : 0;
    for (long long t0 = static_cast<long long>(t) * kRows; t0 < own; t0 += kThreads * kRows) {
        // their sequences and positions, then the pages of all of them at once, then their slots
        int b = t0 < all_rows ? first_above(cu + 1, in.B, static_cast<int>(t0)) : in.B;
        int p[kRows], s[kRows];
        const int *from[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int at = static_cast<int>(t0) + u;  // behind T it is written nowhere
            p[u] = s[u] = -1;
            from[u] = nullptr;
            while (b < in.B && at >= cu[b + 1])
                ++b;
            if (b >= in.B || at >= rows.T)
                continue;
            const long long had = in.had[b];
            const int before = b > 0 ? until[b - 1] : 0;
            const int n = cu[b + 1] - cu[b];
            // a row has a sequence with n > 0: it was refused if it did not fit, or its pages did not
            if (had + n > cap || cu[b + 1] > rows.T || (until[b] > before && until[b] > ring.free))
                continue;
            p[u] = static_cast<int>(had) + at - cu[b];
            const int column = p[u] >> log2_page, old = static_cast<int>(pages_of(had, log2_page));
            from[u] = column < old ? table + b * table_stride + column
                                   : pool.ring + place(pool.size, ring.begin, before + column - old);
        }
        int page[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u)
            page[u] = from[u] ? *from[u] : 0;
#pragma unroll
        for (int u = 0; u < kRows; ++u)
            if (from[u]) {
                if (page[u] >= 0 && page[u] < pool.size)
                    s[u] = (page[u] << log2_page) + (p[u] & ((1 << log2_page) - 1));
                else
                    bad = true;
            }
        rows.write(t0, p, s);
    }
    if (bad)
        atomicOr(status, kStatusBounds);
    if (t == kThreads - 1) {  // which has read the counts, if they are the ones that are written
        const long long counts0 = pool.counts[0], counts1 = pool.counts[1];
        pool.out[0] = counts0 + taken;
        pool.out[1] = counts1;
    }
}

// The rows of more than kOwnRows, a warp 32 * kRows of them: from cu_seqlens, ends (a
// sequence with new rows and no new end was refused) and the page table.
__global__ void __launch_bounds__(kRowThreads)
    fa_cache_rows_kernel(Lengths in, const int *table, long long table_stride, int num_pages, const int *cu_seqlens,
                         const int *ends, Rows rows, unsigned int *status)
{
    cache::wait_ahead();
    cache::let_next();
    const int lane = threadIdx.x & 31;
    const long long w0 = (static_cast<long long>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5)) * (32 * kRows);
    if (w0 >= rows.T)
        return;
    const int *until = cu_seqlens + 1;  // until[b]: the first row behind sequence b
    // the sequences of the warp's first row and of its last: 32 borders a look
    int lo[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int x = static_cast<int>(min(w0 + (i ? 32 * kRows - 1 : 0), static_cast<long long>(rows.T) - 1));
        int n = in.B;  // first above x in [lo, lo + n], as first_above
        while (n > 0) {
            const int step = (n + 31) / 32, at = min(lane * step + step - 1, n - 1);
            const unsigned above = __ballot_sync(0xffffffffu, until[lo[i] + at] > x);
            if (!above) {
                lo[i] += n;
                break;
            }
            const int first = __ffs(above) - 1;  // the border is in this lane's step, before its last
            const int left = first * step, right = min(left + step - 1, n - 1);
            lo[i] += left;
            n = right - left;
        }
    }
    const long long t0 = w0 + lane * kRows;
    if (t0 >= rows.T)
        return;
    int b = lo[0] + first_above(until + lo[0], lo[1] - lo[0], static_cast<int>(t0));
    int p[kRows], s[kRows];
    const int *from[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const int at = static_cast<int>(t0) + u;
        p[u] = s[u] = -1;
        from[u] = nullptr;
        while (b < in.B && at >= until[b])
            ++b;
        if (b >= in.B || at >= rows.T)
            continue;
        const int had = in.had[b];
        if (ends[b] == had)
            continue;
        p[u] = had + at - cu_seqlens[b];
        from[u] = table + b * table_stride + (p[u] >> in.log2_page);
    }
    int page[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u)
        page[u] = from[u] ? *from[u] : 0;
    bool bad = false;
#pragma unroll
    for (int u = 0; u < kRows; ++u)
        if (from[u]) {
            if (page[u] >= 0 && page[u] < num_pages)
                s[u] = (page[u] << in.log2_page) + (p[u] & ((1 << in.log2_page) - 1));
            else
                bad = true;
        }
    rows.write(t0, p, s);
    if (bad)
        atomicOr(status, kStatusBounds);
}

__global__ void __launch_bounds__(kThreads)
    fa_cache_trim_kernel(Pool pool, Lengths in, const int *table, long long table_stride, int max_pages,
                         unsigned int *status)
{
    extern __shared__ int smem[];
    __shared__ long long warps[kThreads / 32];
    __shared__ Ring ring;
    __shared__ int back_all;
    int *until = smem;
    const int t = threadIdx.x;
    const int log2_page = in.log2_page;
    const long long cap = static_cast<long long>(max_pages) << log2_page;
    cache::wait_ahead();
    cache::let_next();
    if (t == kThreads - 1) {
        ring.read(pool);
        back_all = 0;
    }
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
    const int room = ring.bad ? 0 : pool.size - ring.free;
    bool bad = t == 0 && ring.bad;
    for (int b = b0; b < b1; ++b) {
        const long long n = gives(b);
        pages += max(0ll, n);
        until[b] = up_to(pages);
        if (n > 0 && pages <= room)
            atomicMax(&back_all, until[b]);
        bad |= n < 0 || (n > 0 && pages > room);
    }
    __syncthreads();
    const int back = back_all;
    for (int j = t; j < back; j += kThreads) {
        const int b = first_above(until, in.B, j);
        const int before = b > 0 ? until[b - 1] : 0;
        const int page = table[b * table_stride + pages_of(in.other[b], log2_page) + (j - before)];
        bad |= page < 0 || page >= pool.size;
        pool.ring[place(pool.size, ring.end, j)] = page;
    }
    if (bad)
        atomicOr(status, kStatusBounds);
    if (t == kThreads - 1) {
        const long long counts0 = pool.counts[0], counts1 = pool.counts[1];
        pool.out[0] = counts0;
        pool.out[1] = counts1 + back;
    }
}

}  // namespace pages
}  // namespace fa
