// fa_cache4_decode_kernel.cuh -- decoding attention over the 4-bit paged cache on
// sm_103a: O = softmax(scale q K^T) V over the keys of a sequence.
//
// Built as the one over the 8-bit cache (fa_cache_decode_kernel.cuh): units of a stage's
// keys dealt out in equal runs to a persistent grid, one warp that copies, four that
// compute with mma.m16n8k16 on fp16, keys as rows and query rows as columns, parts
// merged by fa_cache_combine_kernel.  (Many short segments of up to 8 rows:
// fa_cache4_short_kernel.cuh; more than 16 rows a head, or 32, unless many and short:
// fa_cache4_tc_kernel.cuh.)  What differs:
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
//    ring (61.0 -> 58.4 us; d = 96 and 64 up to 5 %
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

#include "fa_cache4_run.cuh"
#include "fa_cache4_running.cuh"

namespace fa {
namespace cache4 {

// As DecCfg of the 8-bit cache, for warps of ROWS query rows.
template <int D, int ROWS>
struct Dec4Cfg {
    static constexpr int D_ = D;
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

    Run run_of;
    if (!find_run<F>(w, run_of))
        return;
    const int box = 1 << w.log2_box, box_bytes = box * (D / 8 * 9);
    if (warp == F::WARPS) {
        load_run<F>(w, run_of, sbase, meta, sbase + F::BAR_OFF, abort_flag);
        return;
    }

    // ---------------- the warps that compute ----------------
    const int g = lane >> 2, c = lane & 3;
    const int key_warps = F::WARPS / w.row_warps;
    const int wk = warp % key_warps, wr = warp / key_warps;
    static_assert(R::KW * 512 <= 8 * F::OROW * 4, "sixteen rows of Q fit the merge area");
    R run(lane, sbase + F::MERGE_OFF + warp * (8 * F::OROW * 4) + lane * 16);
    int head = 0, group = 0;
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
