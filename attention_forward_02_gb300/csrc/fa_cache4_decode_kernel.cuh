// fa_cache4_decode_kernel.cuh -- decoding attention over the 4-bit paged cache on
// sm_103a: O = softmax(scale q K^T) V over the keys of a sequence.
//
// Built as the one over the 8-bit cache (fa_cache_decode_kernel.cuh): units of a stage's
// keys dealt out in equal runs to a persistent grid, one warp that copies, four that
// compute with mma.m16n8k16 on fp16, keys as rows and query rows as columns, parts
// merged by fa_cache_combine_kernel.  (Many short segments: fa_cache4_short_kernel.cuh.)  What
// differs:
//  - A page and head is one block of bytes, so that a copy is one bulk copy (four where a
//    page is larger than a stage).  It is not swizzled: of a tile's 16 rows, row r stands for
//    the key r ^ (r >> 2 & 1), and then the reads of K are free of bank conflicts and those
//    of V at most two-way.
//  - Codes become fp16 by cvt (two at a time), times their scale: both exact.  For V the codes
//    of two keys are put side by side first, even channels in one word and odd in another.
//    Up to four rows a head this is not needed: the eight columns of a product are then four
//    rows twice, and the two channels that a byte holds two terms of it, each with the key's
//    weight in one half of the columns and 0 in the other (PAIRS; 124 -> 113 us for the
//    64 sequences below).
//  - Scales belong to keys and channels, so none enters the softmax: P's reference is a plain
//    running maximum (2^kAim under it, as there).
//  - A segment's begin and end (its queries' rows, the merge of its warps) cost a block about
//    as much as OPEN units, and count so when the runs are dealt out: the slowest block was
//    12 to 26 % over the mean before (OPEN 0, 1, 2, 3: 130, 128, 125, 128 us for those 64
//    sequences, 70, 67, 66, 66 for the 16 of 16 rows).
//  - Two stages of 128 keys hide what latency there is (three: 113.5 us, two 115.1), so the
//    16-row warps of d = 128, two blocks an SM, take stages of 256: half the visits to the
//    ring (61.0 -> 58.4 us; 32 and 64 rows a head as before, and d = 96 and 64 up to 5 %
//    slower in short contexts, so there not).
//
// What bounds it: instructions.  16 keys of d = 128 are 2,304 bytes, for which HBM takes some
// 100 clocks of an SM.  A tile costs a warp 260 instructions (four rows) to 330 (sixteen),
// and pipes that take two clocks an instruction: 64 conversions on that of logic, 64
// scalings on the multiplying one, and products of 8.4 clocks, 16 (32) a tile; the three
// overlap only in part (32 + 32 + 8 of them take 105 clocks of a scheduler, each kind alone
// 62).  Without copies the 64 sequences took 122 us where they took 124 with them.
//
// Measured on the GPU, d = 128, 8 KV heads: 64 sequences of up to 16,384 keys, 4 rows a head,
// 675 MB: 113 us, 6.0 TB/s, 88 % of the measured copy rate; 16 of them 41 (4 rows), 45 (8)
// and 58 (16, two blocks an SM: 168 registers); one of 131,072 keys, 8 rows, 151 MB: 37;
// some 10 us of these are start, merge and end.  d = 64, 32 heads of a row, 8 x up to 8,000
// keys, 78 MB: 25; d = 96 and 32: 53 and 36 % of the copy rate, the softmax's instructions
// being the same for fewer bytes.
#pragma once

#include "fa_cache4_running.cuh"

namespace fa {
namespace cache4 {

using cache::kFirst;
using cache::kHeadPart;
using cache::kLast;
using cache::kTailPart;

// As DecCfg of the 8-bit cache, for warps of ROWS query rows.
template <int D, int ROWS>
struct Dec4Cfg {
    static constexpr int LOG2_STEP = D == 128 && ROWS == 16 ? 8 : 7;
    static constexpr int STEP = 1 << LOG2_STEP;
    static constexpr int SUBS = STEP / kTile;
    static constexpr int STAGE = STEP * D / 8 * 9;  // bytes
    static constexpr int WARPS = 4;                 // that compute
    static constexpr int THREADS = 32 * (WARPS + 1);
    static constexpr int BLOCKS = D == 32 ? 4 : D >= 96 && ROWS == 16 ? 2 : 3;  // an SM
    static constexpr int STAGES = D == 128 ? (ROWS == 16 ? 2 : 3) : D == 96 && BLOCKS == 3 ? 4 : 5;
    static constexpr int J = 2;                     // tiles of a warp at once
    static constexpr int OPEN = 256 / STEP;         // units that a segment's begin and end cost
    static_assert(SUBS >= J * WARPS, "every warp has tiles of a stage");
    static constexpr int OROW = D + 4;
    static constexpr int META_OFF = STAGES * STAGE;
    static constexpr int MERGE_OFF = META_OFF + STAGES * 32;
    static constexpr int ML_OFF = MERGE_OFF + WARPS * 8 * OROW * 4;
    static constexpr int BAR_OFF = ML_OFF + WARPS * 8 * 8;
    static constexpr int FLAG_OFF = BAR_OFF + 16 * STAGES + 16;
    static constexpr int SMEM = FLAG_OFF + 16 + 16 * WARPS + 128;  // and room to align the ring
    static_assert(STAGE % 128 == 0, "alignment of the ring");
};

// What the computing warps know of a stage: flags, with a bit from kBoxes on for every box that
// was copied, and the unit's number within the sequence; b .. group with kFirst.
struct __align__(16) Stage4 {
    int flags, unit, b, head, group, pad[3];
};
static_assert(sizeof(Stage4) == 32, "stage record");
constexpr int kEnd = 32;  // the block's last stage
constexpr int kBoxes = 8;  // number of the first box's bit

template <int D, int ROWS, typename T>
__global__ void __launch_bounds__(Dec4Cfg<D, ROWS>::THREADS, Dec4Cfg<D, ROWS>::BLOCKS)
    fa_cache4_decode_kernel(const __grid_constant__ Work w, T *__restrict__ out, float *__restrict__ lse)
{
    using F = Dec4Cfg<D, ROWS>;
    constexpr int S = F::STAGES, J = F::J;
    using R = Running<D, ROWS, T>;
    constexpr int NT = R::NT;
    constexpr int VW = D / 32;  // fours of channels of a thread
    extern __shared__ uint8_t smem_raw[];
    __shared__ long long scan[F::WARPS + 1];
    __shared__ long long begin[2];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 127u) & ~127u;
    uint8_t *smem = smem_raw + (sbase - raw);
    auto full = [&](int s) -> uint32_t { return sbase + F::BAR_OFF + 8u * s; };
    auto empty = [&](int s) -> uint32_t { return sbase + F::BAR_OFF + 8u * (S + s); };
    const uint32_t merged = sbase + F::BAR_OFF + 16u * S;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + F::FLAG_OFF);
    Stage4 *meta = reinterpret_cast<Stage4 *>(smem + F::META_OFF);
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int rows_block = 8 * NT * w.row_warps;
    const int log2_page = w.cache.log2_page;

    if (t == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), F::WARPS);
        }
        mbar_init(merged, F::WARPS);
        *abort_flag = 0;
        fence_mbar_init();
    }
    cache::wait_ahead();
    cache::let_next();

    // ---- this block's run of units ----
    int left = 0;       // its length
    int b;              // its first sequence
    long long off = 0;  // ... and where in that sequence it begins
    int head = 0, group = 0;  // with `whole`, its segment
    if (w.whole) {
        int x = blockIdx.x;
        group = x % w.groups;
        x /= w.groups;
        head = x % w.cache.heads;
        b = x / w.cache.heads;
        if (t == 0 && group == 0 && head == 0)
            w.batch.check_length(b, log2_page);
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
        for (int x = 0; x < F::WARPS + 1; ++x) {
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
            return;
        b = static_cast<int>(begin[0]);
        off = begin[1];
        left = static_cast<int>(min(share, total - first_unit));
    }

    const int box = 1 << w.log2_box, box_bytes = box * (D / 8 * 9);
    if (warp == F::WARPS) {
        // ---------------- the warp that loads ----------------
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
        const int log2_boxes = F::LOG2_STEP - w.log2_box;  // boxes of a stage: 1 to 8
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
                if (done >= S && !(ok = wait_warp(empty(s), phase ^ 1u, abort_flag)))
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
                        bulk_load(dst, src, box_bytes, full(s), policy);
                    } else {  // a part of the page: rows of its four arrays
                        const int y = key & (w.cache.page - 1);
                        const uint32_t half = box_bytes / 2, from = static_cast<uint32_t>(page_bytes / 2);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            bulk_load(dst + i * half, src + i * from + y * (D / 2), box * (D / 2), full(s), policy);
                            bulk_load(dst + i * half + box * (D / 2), src + i * from + w.cache.page * (D / 2) + y * (D / 16),
                                      box * (D / 16), full(s), policy);
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
                    mbar_arrive_expect_tx(full(s), __popc(copied) * box_bytes);
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
        // the computing warps wait for every copy; after a failed wait this one does
        if (!ok)
            for (int x = 0; x < S; ++x)
                if (done > x)
                    drain_bounded(full(x), ((done - 1 - x) / S) & 1);
        return;
    }

    // ---------------- the warps that compute ----------------
    const int g = lane >> 2, c = lane & 3;
    const int key_warps = F::WARPS / w.row_warps;
    const int wk = warp % key_warps, wr = warp / key_warps;
    static_assert(R::KW * 512 <= 8 * F::OROW * 4, "sixteen rows of Q fit the merge area");
    R run(lane, sbase + F::MERGE_OFF + warp * (8 * F::OROW * 4) + lane * 16);
    int4 *segment = reinterpret_cast<int4 *>(smem + F::FLAG_OFF + 16) + warp;  // b, head, group
    uint32_t merges = 0;
    // a barrier of the computing warps whose wait is bounded
    auto meet = [&]() -> bool {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(merged);
        return wait_warp(merged, merges++ & 1u, abort_flag);
    };
    // where in a stage a tile's codes and scales of K begin; those of V lie half a box behind
    auto place = [&](int sub) -> uint2 {
        const int row = sub * kTile, in_box = row & (box - 1);
        const uint32_t at = (row >> w.log2_box) * box_bytes;
        return make_uint2(at + in_box * (D / 2), at + box * (D / 2) + in_box * (D / 16));
    };
    static_assert(NT > 1 || F::SUBS == J * F::WARPS, "with eight rows a block a warp has the same tiles of every stage");
    uint2 own[J];  // ... these
#pragma unroll
    for (int j = 0; j < J; ++j)
        own[j] = place(wk * J + j);
    const unsigned all_boxes = (1u << (F::STEP >> w.log2_box)) - 1u;
    const uint32_t half = box_bytes / 2;
    const uint32_t k_codes = run.key_row * (D / 2) + c * (D / 8), k_scales = run.key_row * (D / 16) + k_scale_offset<D>(c);
    uint32_t v_codes[2], v_scales[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        v_codes[r] = half + run.v_row[r] * (D / 2) + v_code_offset<D>(g);
        v_scales[r] = half + run.v_row[r] * (D / 16) + v_scale_offset<D>(g);
    }
    int slot = S - 1;
    uint32_t phase = 1;
    for (int flags = 0; !(flags & kEnd);) {
        if (++slot == S)
            slot = 0;
        if (slot == 0)
            phase ^= 1u;
        if (!wait_warp(full(slot), phase, abort_flag))
            return;
        const Stage4 *info = meta + slot;
        const int2 what = *reinterpret_cast<const int2 *>(&info->flags);
        flags = what.x;

        if (flags & kFirst) {
            const int b_seg = info->b;
            head = info->head;
            group = info->group;
            if (lane == 0)
                *segment = make_int4(b_seg, head, group, 0);
            __syncwarp();
            run.open(w, b_seg, head, group * rows_block + wr * (8 * NT), w.batch.length(b_seg, log2_page));
        }

        const uint32_t base = sbase + slot * F::STAGE;
        for (int set = wk; set < F::SUBS / J; set += key_warps) {
            // J tiles at once: one look at the reference, and twice the independent work
            const int sub0 = set * J, first = (what.y << F::LOG2_STEP) + sub0 * kTile;
            const bool last_set = NT == 1 || set + key_warps >= F::SUBS / J;
            int key0[J];
#pragma unroll
            for (int j = 0; j < J; ++j)
                key0[j] = first + j * kTile;
            bool masked = first + J * kTile > run.least, some = first < run.most;
            if (static_cast<unsigned>(flags) >> kBoxes != all_boxes) {  // the end, or a page with a bad number
                masked = true;
                some = false;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    if (!(flags >> (kBoxes + ((sub0 + j) * kTile >> w.log2_box)) & 1))
                        key0[j] = kNoKey;
                    some |= key0[j] < run.most;
                }
            }
            if (!some) {
                if (last_set) {
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(empty(slot));
                }
                continue;
            }
            uint32_t codes[J], scales[J];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const uint2 at = NT == 1 ? own[j] : place(sub0 + j);
                codes[j] = base + at.x;
                scales[j] = base + at.y;
            }
            float e[J][NT][4];
            {
                uint32_t kw[J][2][D / 32], ks[J][2][R::KS];
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        load_k<D>(codes[j] + k_codes + r * (8 * D / 2), scales[j] + k_scales + r * (8 * D / 16), kw[j][r],
                                  ks[j][r]);
                run.template scores<J>(kw, ks, e);
            }
            uint32_t pb[J][NT][2];
            run.template weights<J>(e, key0, masked, pb);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                uint32_t vw[4][R::VX], vs[4][R::VX];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    load_v<D>(codes[j] + v_codes[r & 1] + (r >> 1) * (8 * D / 2),
                              scales[j] + v_scales[r & 1] + (r >> 1) * (8 * D / 16), g, vw[r], vs[r]);
                if (j == J - 1 && last_set) {  // the stage's bytes are in registers
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(empty(slot));
                }
                run.values(vw, vs, pb[j], key0[j], masked);
            }
        }

        if (flags & kLast) {
            // ---- merge the warps of each row group, eight rows a warp at a time;
            // write the rows, or the block's part ----
            float *mo = reinterpret_cast<float *>(smem + F::MERGE_OFF);
            float *mm = reinterpret_cast<float *>(smem + F::ML_OFF), *ml = mm + F::WARPS * 8;
            const int b_seg = segment->x;
            head = segment->y;
            group = segment->z;
            const bool part = flags & (kHeadPart | kTailPart);
            const long long place = 2ll * blockIdx.x + (flags & kTailPart ? 1 : 0);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float sum = run.l[nt][u];
                    sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                    const int row = warp * 8 + 2 * c + u;
                    if (g == 0) {
                        mm[row] = run.unset >> (2 * nt + u) & 1u ? -INFINITY : run.m[nt][u];
                        ml[row] = sum;
                    }
                    if constexpr (R::PAIRS) {
                        // rows 2 (c & 1), + 1; channels: those of v_column, first ones at c < 2, second at c >= 2
                        float *to = mo + (warp * 8 + 2 * (c & 1) + u) * F::OROW + (c >> 1);
#pragma unroll
                        for (int x = 0; x < VW; ++x) {
                            to[cache::v_column<D>(g, x)] = run.acc[x][0][u];
                            to[cache::v_column<D>(g, x) + 2] = run.acc[x][0][u + 2];
                        }
                    } else {
#pragma unroll
                        for (int x = 0; x < VW; ++x)
                            *reinterpret_cast<float4 *>(mo + row * F::OROW + cache::v_column<D>(g, x)) =
                                make_float4(run.acc[2 * x][nt][u], run.acc[2 * x][nt][u + 2], run.acc[2 * x + 1][nt][u],
                                            run.acc[2 * x + 1][nt][u + 2]);
                    }
                }
                if (!meet())
                    return;
                for (int x = t; x < 8 * w.row_warps * (D / 4); x += 32 * F::WARPS) {
                    const int r8 = x / (D / 4), d = 4 * (x % (D / 4));
                    const int row = r8 / 8 * (8 * NT) + nt * 8 + r8 % 8;  // of the block
                    const int abs_row = group * rows_block + row;
                    if (abs_row >= w.R)
                        continue;
                    const int from = (r8 / 8) * key_warps * 8 + r8 % 8;  // of its first warp
                    float f[F::WARPS], top = -INFINITY, sum = 0.f;
#pragma unroll
                    for (int y = 0; y < F::WARPS; ++y) {
                        f[y] = y < key_warps ? mm[from + y * 8] : -INFINITY;
                        top = fmaxf(top, f[y]);
                    }
                    const float ref = top == -INFINITY ? 0.f : top;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int y = 0; y < F::WARPS; ++y)
                        if (y < key_warps) {
                            const float4 z = *reinterpret_cast<const float4 *>(mo + (from + y * 8) * F::OROW + d);
                            f[y] = cache::ex2(f[y] - ref);
                            o.x = fmaf(z.x, f[y], o.x);
                            o.y = fmaf(z.y, f[y], o.y);
                            o.z = fmaf(z.z, f[y], o.z);
                            o.w = fmaf(z.w, f[y], o.w);
                            sum = fmaf(ml[from + y * 8], f[y], sum);
                        }
                    if (part) {
                        const long long pr = place * rows_block + row;
                        *reinterpret_cast<float4 *>(w.part_o + pr * D + d) = o;
                        if (d == 0) {
                            w.part_m[pr] = top;
                            w.part_l[pr] = sum;
                        }
                    } else {
                        const long long orow = (static_cast<long long>(b_seg) * w.cache.heads + head) * w.R + abs_row;
                        const float inv = sum == 0.f ? 0.f : 1.f / sum;
                        *reinterpret_cast<uint2 *>(out + orow * D + d) = make_uint2(
                            DTypeTraits<T>::pack(o.x * inv, o.y * inv), DTypeTraits<T>::pack(o.z * inv, o.w * inv));
                        if (d == 0 && lse != nullptr)
                            lse[orow] = sum == 0.f ? -INFINITY : (ref + __log2f(sum)) * 0.6931471805599453f;
                    }
                }
                if (!meet())  // the area is free: for the next rows, for the next segment's Q
                    return;
            }
        }
    }
}

}  // namespace cache4
}  // namespace fa
