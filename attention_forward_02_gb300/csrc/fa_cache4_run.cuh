// fa_cache4_run.cuh -- what the kernels of a persistent grid over the 4-bit cache share: a block's
// run of units, and the warp that copies its keys, a unit of F::STEP a stage, into a ring.
#pragma once

#include "fa_cache4_kernel.cuh"
#include "fa_cache_decode_kernel.cuh"

namespace fa {
namespace cache4 {

using cache::kFirst;
using cache::kHeadPart;
using cache::kLast;
using cache::kTailPart;
using cache::Work;

// What the computing warps know of a stage: flags, with a bit from kBoxes on for every box that
// was copied, and the unit's number within the sequence; b .. group with kFirst.
struct __align__(16) Stage4 {
    int flags, unit, b, head, group, pad[3];
};
static_assert(sizeof(Stage4) == 32, "stage record");
constexpr int kEnd = 32;  // the block's last stage
constexpr int kBoxes = 8;  // number of the first box's bit

// A block's run of units.
struct Run {
    int left = 0;              // its length
    int b = 0;                 // its first sequence
    long long off = 0;         // ... and where in that sequence it begins
    int head = 0, group = 0;   // with `whole`, its segment
};

// False if the block has none.  All threads call it; what they wrote to shared memory before is seen
// by all afterwards.
template <typename F>
__device__ __forceinline__ bool find_run(const Work &w, Run &r)
{
    __shared__ long long scan[F::THREADS / 32];
    __shared__ long long begin[2];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int log2_page = w.cache.log2_page;
    if (w.whole) {
        int x = blockIdx.x;
        r.group = x % w.groups;
        x /= w.groups;
        r.head = x % w.cache.heads;
        r.b = x / w.cache.heads;
        if (t == 0 && r.group == 0 && r.head == 0)
            w.batch.check_length(r.b, log2_page);
        __syncthreads();  // the barriers are set
    } else {
        const int each = (w.B + F::THREADS - 1) / F::THREADS;
        const int b0 = min(w.B, t * each), b1 = min(w.B, b0 + each);
        long long sum = 0;
        for (int x = b0; x < b1; ++x)
            sum += cache::units_of_sequence<F::LOG2_STEP, F::OPEN>(w, x);
        long long incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += y;
        }
        if (lane == 31)
            scan[warp] = incl;
        __syncthreads();
        long long total = 0;
        for (int x = 0; x < F::THREADS / 32; ++x) {
            if (x < warp)
                incl += scan[x];
            total += scan[x];
        }
        // longer than a segment's begin, so that every run has a unit (the last one ends with one)
        const long long share = max(F::OPEN + 1ll, (total + gridDim.x - 1) / gridDim.x);
        const long long first_unit = share * blockIdx.x;
        long long at = incl - sum;
        if (blockIdx.x == 0) {
            if (t == 0)
                w.plan[0] = share;
            long long y = at;
            for (int x = b0; x < b1; ++x) {
                w.plan[1 + x] = y;
                w.batch.check_length(x, log2_page);
                y += cache::units_of_sequence<F::LOG2_STEP, F::OPEN>(w, x);
            }
        }
        if (first_unit >= at && first_unit < incl) {
            int x = b0;
            for (; x + 1 < b1; ++x) {
                const long long n = cache::units_of_sequence<F::LOG2_STEP, F::OPEN>(w, x);
                if (first_unit < at + n)
                    break;
                at += n;
            }
            begin[0] = x;
            begin[1] = first_unit - at;
        }
        __syncthreads();
        if (first_unit >= total)
            return false;
        r.b = static_cast<int>(begin[0]);
        r.off = begin[1];
        r.left = static_cast<int>(min(share, total - first_unit));
    }
    return true;
}

// The warp that loads.  sbase: of the ring of F::STAGES stages; full0: barriers of full stages, and
// behind them of empty ones.
template <typename F>
__device__ __forceinline__ void load_run(const Work &w, const Run &r, uint32_t sbase, Stage4 *meta, uint32_t full0,
                                         volatile int *abort_flag)
{
    constexpr int S = F::STAGES, D = F::D_;
    const int lane = threadIdx.x & 31;
    const int log2_page = w.cache.log2_page;
    const int box = 1 << w.log2_box, box_bytes = box * (D / 8 * 9);
    int left = r.left, b = r.b, head = r.head, group = r.group;
    const long long off = r.off;
    int len = 0, units = 0, unit = 0;
    auto open_sequence = [&]() {
        len = b < w.B ? w.batch.length(b, log2_page) : 0;
        units = cache::units_of<F::LOG2_STEP>(w, len, 0);
    };
    open_sequence();
    if (w.whole) {
        units = left = max(1, units);  // without keys it has a unit all the same, and writes its rows in it
    } else {
        // off < (units + OPEN) * heads * groups here: 32 bits hold it unless a sequence's work is vast
        const int span = units + F::OPEN;
        const int seg = off >> 31 ? static_cast<int>(off / span) : static_cast<int>(off) / span;
        head = seg / w.groups;
        group = seg % w.groups;
        unit = static_cast<int>(off - static_cast<long long>(seg) * span) - F::OPEN;
        left += min(unit, 0);  // what is left of the segment's begin
        unit = max(unit, 0);
    }
    const int log2_boxes = F::LOG2_STEP - w.log2_box;  // boxes of a stage: 1 to 16
    const int batch_units = 32 >> log2_boxes;
    const size_t page_bytes = static_cast<size_t>(w.cache.page) * (D / 8 * 9);
    const uint64_t policy = l2_policy_evict_first();
    bool opened = true, ok = true;  // opened: the next unit is this block's first of its segment
    bool begun = unit == 0;         // this block has the segment's first unit
    const unsigned stage_lanes = (1u << (1 << log2_boxes)) - 1u;
    int done = 0, s = 0;
    uint32_t phase = 0;  // of the ring's round
    while (left > 0 && ok) {
        // lane l: page of the l-th of the next 32 boxes of this segment
        const int here = min(min(batch_units, units - unit), left);
        if (here <= 0)  // lengths that changed under the call: the other warps' waits will give up
            break;
        const int key = (unit << F::LOG2_STEP) + lane * box;
        int p = -1;
        if ((lane >> log2_boxes) < here && key < len) {
            p = w.batch.page(b, key >> log2_page);
            if (p < 0)
                w.batch.bad();
        }
        const uint8_t *src = w.cache.k + (static_cast<size_t>(max(p, 0)) * w.cache.heads + head) * page_bytes;
        const unsigned alive = __ballot_sync(0xffffffffu, p >= 0);
        for (int u = 0; u < here; ++u, ++done) {
            if (done >= S && !(ok = wait_warp(full0 + 8u * (S + s), phase ^ 1u, abort_flag)))
                break;
            const int first_lane = u << log2_boxes;
            const bool mine = (lane >> log2_boxes) == u;
            --left;
            const bool last = left == 0 || (unit + 1 == units && left <= F::OPEN);
            const bool ended = unit + 1 == units || last;
            // the copies first (their bytes may arrive before they are expected: the phase
            // waits for the arrival below), then the record
            if (mine && p >= 0) {
                const uint32_t dst = sbase + s * F::STAGE + (lane - first_lane) * box_bytes;
                if (w.cache.page == box) {
                    bulk_load(dst, src, box_bytes, full0 + 8u * s, policy);
                } else {  // a part of the page: rows of its four arrays
                    const int y = key & (w.cache.page - 1);
                    const uint32_t half = box_bytes / 2, from = static_cast<uint32_t>(page_bytes / 2);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        bulk_load(dst + i * half, src + i * from + y * (D / 2), box * (D / 2), full0 + 8u * s, policy);
                        bulk_load(dst + i * half + box * (D / 2), src + i * from + w.cache.page * (D / 2) + y * (D / 16),
                                  box * (D / 16), full0 + 8u * s, policy);
                    }
                }
            }
            int flags = (opened ? kFirst : 0) | (ended ? kLast : 0) | (last ? kEnd : 0);
            // does this block have the segment from its first to its last unit?
            if (ended && !begun)
                flags |= kHeadPart;  // it began before this block's run
            else if (ended && unit + 1 < units)
                flags |= kTailPart;
            const unsigned copied = alive >> first_lane & stage_lanes;
            if (lane == 0) {
                Stage4 *m = meta + s;
                *reinterpret_cast<int2 *>(&m->flags) = make_int2(flags | static_cast<int>(copied << kBoxes), unit);
                if (opened) {
                    m->b = b;
                    m->head = head;
                    m->group = group;
                }
                mbar_arrive_expect_tx(full0 + 8u * s, __popc(copied) * box_bytes);
            }
            opened = ended;
            ++unit;
            if (++s == S) {
                s = 0;
                phase ^= 1u;
            }
        }
        if (unit == units && (left -= F::OPEN) > 0) {  // on to the next segment
            unit = 0;
            begun = true;
            if (++group == w.groups) {
                group = 0;
                if (++head == w.cache.heads) {
                    head = 0;
                    do {
                        ++b;
                        open_sequence();
                    } while (units == 0 && b < w.B);
                }
            }
        }
    }
    // the block does not end before its copies, whatever made the other warps leave
    for (int x = 0; x < S; ++x)
        if (done > x)
            drain_bounded(full0 + 8u * x, ((done - 1 - x) / S) & 1);
}

}  // namespace cache4
}  // namespace fa
