// fa_cache4_short_kernel.cuh -- decoding attention over the 4-bit paged cache where many
// segments, a sequence and KV head each, are short: a warp takes a whole one.
//
// The kernel of fa_cache4_decode_kernel.cuh pays for every segment that a block begins and
// ends about what OPEN units cost (2.8 us of a block: the queries' rows, the first copies, the
// merge of four warps, the parts and their launch), which for a few hundred keys is most of
// the time.  Here nothing is shared: the four warps of a block have a segment each, copy its
// keys themselves into a ring of two stages of 32 keys, merge with nobody and write the rows.
// 16 warps an SM take their turns at waiting.
//
// What bounds it: a warp's own chain, 0.85 us for 32 keys (copy, products, softmax, products),
// while segments are few; instructions, as there, when the SMs are full.  Stages of three or
// four change little (2 % slower: fewer bytes of shared memory are L1); K and V read straight
// into registers without a copy, the next 32 keys ahead, took 10 to 30 % longer.
//
// Measured on the GPU, d = 128, 8 KV heads of 4 rows, up to 300 keys a sequence: 64 sequences
// 11.4 us (13.8 by the other kernel), 128 13.9 (19.2), 512 31.4 (53.0: 102 MB, 48 % of the
// measured copy rate); 512 of 7 keys 11.1 (36.1), 64 of 7 keys 3.7 (9.9).
#pragma once

#include "fa_cache4_running.cuh"

namespace fa {
namespace cache4 {

template <int D, int ROWS>
struct Short4Cfg {
    static constexpr int WARPS = 4, THREADS = 32 * WARPS;
    static constexpr int BLOCKS = 4;           // an SM
    static constexpr int J = 2;                // tiles at once: a stage
    static constexpr int STEP = J * kTile;
    static constexpr int LOG2_STEP = 5;
    static constexpr int STAGES = 2;           // of a warp
    static constexpr int STAGE = STEP * D / 8 * 9;
    static constexpr int BAR_OFF = WARPS * STAGES * STAGE;
    static constexpr int FLAG_OFF = BAR_OFF + WARPS * STAGES * 8;
    static constexpr int SMEM = FLAG_OFF + 16;
    static_assert(1 << LOG2_STEP == STEP && STAGE % 16 == 0 && J * STAGES <= 32, "bookkeeping of stages");
};

template <int D, int ROWS, typename T>
__global__ void __launch_bounds__(Short4Cfg<D, ROWS>::THREADS, Short4Cfg<D, ROWS>::BLOCKS)
    fa_cache4_short_kernel(const __grid_constant__ Work w, T *__restrict__ out, float *__restrict__ lse)
{
    using F = Short4Cfg<D, ROWS>;
    using R = Running<D, ROWS, T>;
    constexpr int J = F::J, S = F::STAGES;
    static_assert(R::NT == 1, "a tile of eight columns");
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t ring = sbase + warp * (S * F::STAGE);
    auto full = [&](int s) -> uint32_t { return sbase + F::BAR_OFF + 8u * (warp * S + s); };
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + F::FLAG_OFF);
    const long long segment = static_cast<long long>(blockIdx.x) * F::WARPS + warp;
    const int b = static_cast<int>(segment / w.cache.heads), head = static_cast<int>(segment % w.cache.heads);
    if (lane < S)
        mbar_init(full(lane), 1);
    if (threadIdx.x == 0)
        *abort_flag = 0;
    fence_mbar_init();
    __syncthreads();
    cache::wait_ahead();
    cache::let_next();
    if (b >= w.B)
        return;

    const int log2_page = w.cache.log2_page, page = 1 << log2_page;
    int slot0 = 0;  // lane l: page of the sequence's slot slot0 + l
    int own = w.batch.page(b, lane);
    const int len = w.batch.length(b, log2_page);
    if (lane == 0 && head == 0)
        w.batch.check_length(b, log2_page);
    const auto report = [&]() {
        if (own < 0 && static_cast<long long>(slot0 + lane) << log2_page < len)
            w.batch.bad();
    };
    report();

    // a stage is a part of a page, or two pages of 16
    const int log2_box = min(log2_page, F::LOG2_STEP), box = 1 << log2_box;
    const int box_bytes = box * (D / 8 * 9), page_bytes = page * (D / 8 * 9);
    const uint64_t policy = l2_policy_evict_first();
    unsigned there = 0;  // J bits of each stage: its tiles that were copied
    // Begins to copy the keys from `first` on to stage s.
    const auto copy = [&](int first, int s) {
        if (first >> log2_page >= slot0 + 32) {
            slot0 += 32;
            own = w.batch.page(b, slot0 + lane);
            report();
        }
        const int key = first + (lane << log2_box);
        const int p = __shfl_sync(0xffffffffu, own, key >> log2_page & 31);
        const bool mine = lane < F::STEP >> log2_box && key < len && p >= 0;
        const unsigned copied = __ballot_sync(0xffffffffu, mine);
        if (mine) {
            const uint8_t *src = w.cache.k + (static_cast<size_t>(p) * w.cache.heads + head) * page_bytes;
            const uint32_t dst = ring + s * F::STAGE + lane * box_bytes;
            if (page == box) {
                bulk_load(dst, src, box_bytes, full(s), policy);
            } else {  // a part of the page: rows of its four arrays
                const int y = key & (page - 1);
                const uint32_t half = box_bytes / 2, from = page_bytes / 2;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    bulk_load(dst + i * half, src + i * from + y * (D / 2), box * (D / 2), full(s), policy);
                    bulk_load(dst + i * half + box * (D / 2), src + i * from + page * (D / 2) + y * (D / 16), box * (D / 16),
                              full(s), policy);
                }
            }
        }
        if (lane == 0)
            mbar_arrive_expect_tx(full(s), __popc(copied) * box_bytes);
        unsigned tiles = 0;
#pragma unroll
        for (int j = 0; j < J; ++j)
            tiles |= (copied >> (j * kTile >> log2_box) & 1u) << j;
        there = (there & ~(((1u << J) - 1u) << (J * s))) | tiles << (J * s);
    };
    const int steps = static_cast<int>((static_cast<long long>(len) + F::STEP - 1) >> F::LOG2_STEP);
    int begun = 0;
    for (; begun < min(S, steps); ++begun)
        copy(begun << F::LOG2_STEP, begun);

    R run(lane, 0);
    const int g = run.g, c = run.c;
    run.open(w, b, head, 0, len);
    const uint32_t half = box_bytes / 2;
    uint32_t codes[J], scales[J];  // where in a stage those of a tile begin
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int row = j * kTile, in_box = row & (box - 1);
        codes[j] = (row >> log2_box) * box_bytes + in_box * (D / 2);
        scales[j] = (row >> log2_box) * box_bytes + box * (D / 2) + in_box * (D / 16);
    }
    const uint32_t k_codes = run.key_row * (D / 2) + c * (D / 8), k_scales = run.key_row * (D / 16) + k_scale_offset<D>(c);
    uint32_t v_codes[2], v_scales[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        v_codes[r] = half + run.v_row[r] * (D / 2) + v_code_offset<D>(g);
        v_scales[r] = half + run.v_row[r] * (D / 16) + v_scale_offset<D>(g);
    }
    int s = 0;
    uint32_t phase = 0;
    for (int step = 0; step < steps; ++step) {
        if (!wait_warp(full(s), phase, abort_flag)) {
            // leaves only after its copies have arrived
            for (; step < begun; ++step) {
                drain_bounded(full(s), phase);
                if (++s == S) {
                    s = 0;
                    phase ^= 1u;
                }
            }
            return;
        }
        const int first = step << F::LOG2_STEP;
        const unsigned now = there >> (J * s);
        const uint32_t base = ring + s * F::STAGE;
        int key0[J];
#pragma unroll
        for (int j = 0; j < J; ++j)
            key0[j] = now >> j & 1 ? first + j * kTile : kNoKey;
        const bool masked = first + F::STEP > run.least || (~now & ((1u << J) - 1u));
        float e[J][1][4];
        {
            uint32_t kw[J][2][D / 32], ks[J][2][R::KS];
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    load_k<D>(base + codes[j] + k_codes + r * (8 * D / 2), base + scales[j] + k_scales + r * (8 * D / 16),
                              kw[j][r], ks[j][r]);
            run.template scores<J>(kw, ks, e);
        }
        uint32_t pb[J][1][2];
        run.template weights<J>(e, key0, masked, pb);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            uint32_t vw[4][R::VX], vs[4][R::VX];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                load_v<D>(base + codes[j] + v_codes[r & 1] + (r >> 1) * (8 * D / 2),
                          base + scales[j] + v_scales[r & 1] + (r >> 1) * (8 * D / 16), g, vw[r], vs[r]);
            if (j == J - 1) {  // the stage's bytes are in registers
                __syncwarp();
                if (begun < steps)
                    copy(begun++ << F::LOG2_STEP, s);
            }
            run.values(vw, vs, pb[j], key0[j], masked);
        }
        if (++s == S) {
            s = 0;
            phase ^= 1u;
        }
    }

    const long long row0 = (static_cast<long long>(b) * w.cache.heads + head) * w.R;
    float inv[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        float sum = run.l[0][u];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const bool none = run.unset >> u & 1u;
        inv[u] = sum == 0.f ? 0.f : 1.f / sum;
        const int row = 2 * c + u;
        if (lse != nullptr && g == 0 && row < w.R)
            lse[row0 + row] = sum == 0.f ? -INFINITY : ((none ? 0.f : run.m[0][u]) + __log2f(sum)) * 0.6931471805599453f;
    }
#pragma unroll
    for (int x = 0; x < D / 32; ++x) {
        const int d = cache::v_column<D>(g, x);
        if constexpr (R::PAIRS) {
            // lanes c and c ^ 2 have every other of four channels, of two rows: each takes a row
            const bool second = c >= 2;
            const float(&a)[4] = run.acc[x][0];
            const float lo0 = a[0] * inv[0], lo1 = a[1] * inv[1], hi0 = a[2] * inv[0], hi1 = a[3] * inv[1];
            const float lo = __shfl_xor_sync(0xffffffffu, second ? lo0 : lo1, 2);
            const float hi = __shfl_xor_sync(0xffffffffu, second ? hi0 : hi1, 2);
            const int row = 2 * (c & 1) + (second ? 1 : 0);
            if (row < w.R)
                *reinterpret_cast<uint2 *>(out + (row0 + row) * D + d) =
                    second ? make_uint2(DTypeTraits<T>::pack(lo, lo1), DTypeTraits<T>::pack(hi, hi1))
                           : make_uint2(DTypeTraits<T>::pack(lo0, lo), DTypeTraits<T>::pack(hi0, hi));
        } else {
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (2 * c + u < w.R)
                    *reinterpret_cast<uint2 *>(out + (row0 + 2 * c + u) * D + d) =
                        make_uint2(DTypeTraits<T>::pack(run.acc[2 * x][0][u] * inv[u], run.acc[2 * x][0][u + 2] * inv[u]),
                                   DTypeTraits<T>::pack(run.acc[2 * x + 1][0][u] * inv[u], run.acc[2 * x + 1][0][u + 2] * inv[u]));
        }
    }
}

}  // namespace cache4
}  // namespace fa
