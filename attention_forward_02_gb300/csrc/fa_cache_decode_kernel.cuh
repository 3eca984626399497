// fa_cache_decode_kernel.cuh -- decoding attention over the 8-bit paged cache
// on sm_103a: O = softmax(scale q K^T) V with K = k_scale * codes, V likewise,
// over all keys of a sequence or over listed pages only.
//
// What bounds it: with up to 16 query rows a KV head the work is 4 * 16 flops
// for two code bytes, far below the ridge, so the time is that of reading the
// codes once from HBM.  All else has to stay under it: per SM about 23 bytes a
// clock arrive, so a warp's 16 keys of d = 128 (4 KB) may take some 170 clocks
// of the SM, issue slots of four schedulers among them.
//
// The products run on the tensor cores in fp16 with fp32 sums: codes convert to
// fp16 exactly, in registers, straight into the operand layout of
// mma.m16n8k16, with keys as the 16 rows and query rows as the 8 columns:
//     S^T = K Q^T   (16 keys x d) (d x 8 queries)
//     O^T += V^T P^T  (d x 16 keys) (16 keys x 8 queries)
// A matrix instruction fed from shared memory would need 8-bit Q and P, or a
// round trip of the converted tile through shared memory; here nothing is
// exchanged between threads but P^T, transposed by movmatrix.  The order of d
// inside the first product, and of the rows of O^T in the second, is free, so a
// thread takes consecutive bytes of a row: 16-byte shared reads, free of bank
// conflicts under the swizzle that TMA writes (d = 128; a few two-way ones below).
//
// One warp loads: it looks up page numbers and scales, 32 pages at a time, and
// copies 64 keys of K and V a stage (128 at d <= 64) into a ring.  Four warps
// compute, 16 or 32 keys each, or, with more than 8 query rows a head, more keys
// and fewer warps on the same rows.
//
// Query rows are scaled by a power of two to a row maximum in [2^14, 2^15)
// before they become fp16: a bf16 row keeps every bit that fp32 sums would see.
// P is rounded to fp16 (2^-12) as P * v_scale against a reference m that
// includes v_scale's exponent, so that V scales of any size mix, and lies 2^10 under
// the largest one seen (kAim below).  m moves (and O, l are rescaled) only when
// one outgrows it by 2^14.9.
//
// Work is dealt in units of a stage's 64 keys (128 at d <= 64) of one (sequence,
// KV head, row group): the blocks of a persistent grid take equal runs of the
// concatenated units of all sequences, whatever their lengths, which are read
// from device memory.  A run may begin and end inside a segment; those parts (at
// most two a block) go to the workspace as (m, l, O) and fa_cache_combine_kernel
// merges them, in a fixed order.  Where the page table bounds the contexts to a
// few units and there are no more segments than resident blocks, a block takes a
// whole segment instead, and that launch is all.
//
// Measured, whole calls back to back (e4m3, d = 128, 8 KV heads): 64 sequences of
// up to 16,384 keys, 4 rows a head, 1.20 GB: 181 to 184 us, 6.5 TB/s, 96 to 98 % of
// the measured copy rate, DRAM reads 1.2036 GB; one of 131,072 keys, 8 rows,
// 269 MB: 51 us, 77 %, where some 10 us of a call are no streaming (lengths, page
// numbers and scales one after the other, the first copies, the merges): twice the
// keys take 37 us more.  The same at d = 64 with one row a head: 8 x up to 8,000 keys,
// 32 heads, 138 MB take 32 us, 63 %, and as many again 22 more, 93 %.  With 16
// rows a head the instructions bound it: 16 sequences, 340 MB of int8 codes,
// 84 us, 59 %; conversions are over a third of them.
#pragma once

#include "fa_cache_kernel.cuh"

namespace fa {
namespace cache {

constexpr int kDecWarps = 4;      // that compute
constexpr int kDecThreads = 32 * (kDecWarps + 1);
constexpr int kTile = 16;         // keys of one product
constexpr int kMaxSubs = 8;       // tiles of a stage
constexpr int kMaxBlocks = 640;   // of the persistent grid
constexpr int kCombineThreads = 128;
constexpr int kCombineEach = 8;   // parts of a warp under way at once

// A code row of d bytes is held in one or two column parts, each with the TMA
// swizzle of its width: 32, 64, 128, or 64 + 32.
template <int D>
struct DecCfg {
    static constexpr int LOG2_STEP = D <= 64 ? 7 : 6;
    static constexpr int STEP = 1 << LOG2_STEP;               // keys of a stage: a unit of work
    static constexpr int SUBS = STEP / kTile;
    static constexpr int PARTS = D == 96 ? 2 : 1;
    static constexpr int W0 = D == 96 ? 64 : D, W1 = D - W0;  // widths
    static constexpr int HALF = STEP * D;                     // K or V of a stage, bytes
    static constexpr int STAGE = 2 * HALF;
    static constexpr int BLOCKS = D == 32 ? 4 : 3;            // an SM
    static constexpr int RING = D == 32 ? 32768 : 49152;      // bytes
    static constexpr int STAGES = RING / STAGE < 8 ? RING / STAGE : 8;  // 3 at d = 128
    static constexpr int OROW = D + 4;                        // floats of a row of the merge
    static constexpr int RING_OFF = 0;
    static constexpr int META_OFF = STAGES * STAGE;
    static constexpr int MERGE_OFF = META_OFF + STAGES * 192;
    static constexpr int ML_OFF = MERGE_OFF + kDecWarps * 8 * OROW * 4;  // eight rows a warp at a time
    static constexpr int BAR_OFF = ML_OFF + kDecWarps * 8 * 8;
    static constexpr int FLAG_OFF = BAR_OFF + 16 * STAGES + 16;  // full, empty, merge
    static constexpr int SMEM = FLAG_OFF + 16 + 16 * kDecWarps + 1024;  // and room to align the ring
    static_assert(STAGES * STAGE % 16 == 0 && STAGE % 1024 == 0, "alignment of the ring");
};

// What the computing warps know of a stage.
struct __align__(16) TileMeta {
    float k_scale;
    float v_log2, v_inv;  // the V scale's power of two, its exponent and reciprocal
    int key0;             // position of the 16-key tile's first key, or kNoKey
};
struct __align__(16) StageMeta {
    TileMeta tile[kMaxSubs];
    float v_rest[kMaxSubs];  // V scale over its power of two; written with kOddScale
    int flags, b, i, head, group, pad[3];  // b .. group with kFirst
};
static_assert(sizeof(StageMeta) == 192, "stage record");
constexpr int kFirst = 1, kLast = 2, kHeadPart = 4, kTailPart = 8, kOddScale = 16;
constexpr int kNoKey = 0x7FFFFF00;  // behind every context

// P is rounded to fp16, whose 2^-14 .. 65,504 has to hold the largest weight of a row and
// the small ones beside it: an attention sink, a key with nearly all the weight and a
// value near zero, leaves the output to weights of 2^-20 of its own and less.  So the
// reference is put 2^kAim under the largest P * v_scale (its power of two), and moves when
// one has grown to 2^kMost (the V scale's factor over its power of two, below 2, is still
// to come: 2^15.9 < 65,504).  Weights down to 2^-24 of the largest keep all eleven bits,
// those down to 2^-34 some.  A sink of 0.9999 over 4,096 keys, bf16: o off by 1.86e-3 of
// itself (rms), of which its own rounding is 1.84e-3; with the reference at the largest
// one 9.0e-3, and 1.8e-2 where a warp has all keys of a row.  The room left for growth
// decides how often the reference moves: at 16 rows a head (16 x 16,384 keys, int8,
// d = 128) 6 and 8 octaves take 84.0 us, 4.9 take 84.4, 4 85.0, 2 87.0 and 1 88.9; up to
// 8 rows it does not show.
constexpr float kAim = 10.f, kMost = 14.9f;

// Where a thread (g = lane / 4, c = lane % 4) finds its bytes of a 16-key tile in
// a part W bytes wide: of K, 4 words (2 if W = 32) ... of rows g and g + 8; of V,
// W / 32 words of the rows 2 c, 2 c + 1, + 8.  Swizzle of a row of W bytes: its
// 16-byte chunk number XOR bits of the row (TMA's 128-, 64- and 32-byte swizzles).
template <int W>
__device__ __forceinline__ uint32_t k_offset(int g, int c, int x)
{
    if (W == 128)
        return g * 128 + (((2 * c + x) ^ g) << 4);
    if (W == 64)
        return g * 64 + ((c ^ ((g >> 1) & 3)) << 4);
    return g * 32 + (((c >> 1) ^ ((g >> 2) & 1)) << 4) + (c & 1) * 8;
}
template <int W>
__device__ __forceinline__ uint32_t v_offset(int g, int c, int odd)
{
    const int row = 2 * c + odd;
    if (W == 128)
        return row * 128 + ((g ^ row) << 4);
    if (W == 64)
        return row * 64 + (((g >> 1) ^ c) << 4) + (g & 1) * 8;
    return row * 32 + (((g >> 2) ^ (c >> 1)) << 4) + (g & 3) * 4;
}
// Column of a thread's K word s, and of its V word x (each 4 consecutive columns).
template <int D>
__device__ __forceinline__ int k_column(int c, int s)
{
    if (D == 128)
        return 32 * c + 4 * s;
    if (D == 64)
        return 16 * c + 4 * s;
    if (D == 32)
        return 8 * c + 4 * s;
    return s < 4 ? 16 * c + 4 * s : 64 + 8 * c + 4 * (s - 4);
}
template <int D>
__device__ __forceinline__ int v_column(int g, int x)
{
    if (D == 96)
        return x < 2 ? 8 * g + 4 * x : 64 + 4 * g;
    return g * (D / 8) + 4 * x;
}

struct Work {
    Cache cache;
    Batch batch;
    Queries q;
    const int *pages;  // listed pages, or NULL
    int slots;
    int B, R, groups;  // rows of a segment (G Nq, or G with listed pages), row groups
    int row_warps;     // warps along the rows (1, 2, 4), the others along the keys
    bool whole;        // a block a segment, from its first key to its last: nothing to merge
    int log2_box;      // keys of one copy: a page, or a stage if that is smaller
    float scale_log2;
    // workspace: [0] blocks' share, [1 + b] first unit of sequence b; then the parts
    long long *plan;
    float *part_o, *part_m, *part_l;  // [2 blocks][rows][D], [2 blocks][rows]
};

// Units of query i's segment of a sequence of `len` keys (all queries' with no list).
template <int LOG2_STEP>
__device__ __forceinline__ int units_of(const Work &w, int len, int i)
{
    int keys = len;
    if (w.pages) {
        const int n = (context(w.q, len, i) + w.cache.page - 1) >> w.cache.log2_page;
        keys = min(n, w.slots) << w.cache.log2_page;
    }
    return keys > 0 ? ((keys - 1) >> LOG2_STEP) + 1 : 0;
}
// Those of sequence b; a segment that has any counts OPEN more.
template <int LOG2_STEP, int OPEN = 0>
__device__ __forceinline__ long long units_of_sequence(const Work &w, int b)
{
    const int len = w.batch.length(b, w.cache.log2_page);
    long long n = 0;
    for (int i = 0; i < (w.pages ? w.q.Nq : 1); ++i) {
        const int units = units_of<LOG2_STEP>(w, len, i);
        n += units > 0 ? units + OPEN : 0;
    }
    return n * w.cache.heads * w.groups;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <int WORDS>
__device__ __forceinline__ void load_words(uint32_t *w, uint32_t addr)
{
    if (!smem_ok(addr, 4 * WORDS, 4 * WORDS)) {
        for (int i = 0; i < WORDS; ++i)
            w[i] = 0;
        return;
    }
    if constexpr (WORDS == 4)
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(addr)
                     : "memory");
    else if constexpr (WORDS == 2)
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
    else
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void store_pair(uint32_t addr, uint32_t a, uint32_t b)
{
    if (smem_ok(addr, 8, 8))
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

// Bytes of a word that are e4m3 NaN codes, as their top bits.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

struct Maps {
    CUtensorMap k[2], v[2];  // of the column parts
};

template <int D, int NT, int J, typename T, typename C>
__global__ void __launch_bounds__(kDecThreads, DecCfg<D>::BLOCKS)
    fa_cache_decode_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Work w, T *__restrict__ out,
                           float *__restrict__ lse)
{
    using F = DecCfg<D>;
    constexpr int S = F::STAGES;
    constexpr int KW = D / 16;  // words of a key's codes a thread holds = steps of the first product
    constexpr int VW = D / 32;  // words of a key's V a thread holds
    extern __shared__ uint8_t smem_raw[];
    __shared__ long long scan[kDecWarps + 1];
    __shared__ long long begin[2];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (sbase - raw);
    auto full = [&](int s) -> uint32_t { return sbase + F::BAR_OFF + 8u * s; };
    auto empty = [&](int s) -> uint32_t { return sbase + F::BAR_OFF + 8u * (S + s); };
    const uint32_t merged = sbase + F::BAR_OFF + 16u * S;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + F::FLAG_OFF);
    StageMeta *meta = reinterpret_cast<StageMeta *>(smem + F::META_OFF);
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    constexpr int ROWS = 8 * NT;  // query rows a warp
    const int rows_block = ROWS * w.row_warps;

    if (t == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), kDecWarps);
        }
        mbar_init(merged, kDecWarps);
        *abort_flag = 0;
        fence_mbar_init();
    }
    wait_ahead();
    let_next();

    // ---- this block's run of units ----
    int all;      // units of this block
    int b;        // its first sequence
    long long off = 0;  // ... and the unit of that sequence it begins with
    int i = 0, head = 0, group = 0;  // with `whole`, its segment
    if (w.whole) {
        int x = blockIdx.x;
        group = x % w.groups;
        x /= w.groups;
        head = x % w.cache.heads;
        x /= w.cache.heads;
        i = w.pages ? x % w.q.Nq : 0;
        b = w.pages ? x / w.q.Nq : x;
        if (t == 0 && group == 0 && head == 0 && i == 0)
            w.batch.check_length(b, w.cache.log2_page);
        // a segment without keys has a unit all the same, and writes its rows in it
        all = max(1, units_of<F::LOG2_STEP>(w, w.batch.length(b, w.cache.log2_page), i));
        __syncthreads();  // the barriers are set
    } else {
        const int each = (w.B + kDecThreads - 1) / kDecThreads;
        const int b0 = min(w.B, t * each), b1 = min(w.B, b0 + each);
        long long sum = 0;
        for (int x = b0; x < b1; ++x)
            sum += units_of_sequence<F::LOG2_STEP>(w, x);
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
        for (int x = 0; x < kDecWarps + 1; ++x) {
            if (x < warp)
                incl += scan[x];
            total += scan[x];
        }
        const long long share = max(1ll, (total + gridDim.x - 1) / gridDim.x);
        const long long first_unit = share * blockIdx.x;
        long long at = incl - sum;
        if (blockIdx.x == 0) {
            if (t == 0)
                w.plan[0] = share;
            long long y = at;
            for (int x = b0; x < b1; ++x) {
                w.plan[1 + x] = y;
                w.batch.check_length(x, w.cache.log2_page);
                y += units_of_sequence<F::LOG2_STEP>(w, x);
            }
        }
        if (first_unit >= at && first_unit < incl) {
            int x = b0;
            for (; x + 1 < b1; ++x) {
                const long long n = units_of_sequence<F::LOG2_STEP>(w, x);
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
        all = static_cast<int>(min(share, total - first_unit));
    }

    if (warp == kDecWarps) {
        // ---------------- the warp that loads ----------------
        int len = 0, ctx = 0, units = 0, unit = 0;
        auto open_query = [&]() {
            len = b < w.B ? w.batch.length(b, w.cache.log2_page) : 0;
            ctx = w.pages ? context(w.q, len, i) : len;
            units = units_of<F::LOG2_STEP>(w, len, i);
        };
        open_query();
        if (w.whole) {
            units = all;
        } else {
            const int per_unit = w.cache.heads * w.groups;
            while (i + 1 < w.q.Nq && off >= static_cast<long long>(units) * per_unit) {
                off -= static_cast<long long>(units) * per_unit;
                ++i;
                open_query();
            }
            // off < units * heads * groups here: 32 bits hold it unless a sequence's work is vast
            const int seg = off >> 31 ? static_cast<int>(off / units) : static_cast<int>(off) / units;
            head = seg / w.groups;
            group = seg % w.groups;
            unit = static_cast<int>(off - static_cast<long long>(seg) * units);
        }
        const int log2_boxes = F::LOG2_STEP - w.log2_box;  // copies of a stage: 1 to 8
        const int box = 1 << w.log2_box, batch_units = 32 >> log2_boxes;
        const uint64_t policy = l2_policy_evict_first();
        bool opened = true, ok = true;  // opened: the next unit is this block's first of its segment
        const unsigned stage_lanes = (1u << (1 << log2_boxes)) - 1u;
        int done = 0, s = 0;
        uint32_t phase = 0;  // of the ring's round
        while (done < all && ok) {
            // lane l: page and scales of the l-th of the next 32 copies of this segment
            const int here = min(min(batch_units, units - unit), all - done);
            const int key = (unit << F::LOG2_STEP) + lane * box;
            int at = key >> w.cache.log2_page, key0 = key, p = -1;
            float ks = 1.f, vs = 1.f;
            if ((lane >> log2_boxes) < here) {
                if (w.pages) {
                    const int n = (ctx + w.cache.page - 1) >> w.cache.log2_page;
                    const int entry =
                        at < min(n, w.slots)
                            ? w.pages[((static_cast<long long>(b) * w.cache.heads + head) * w.q.Nq + i) * w.slots + at]
                            : -1;
                    if (entry >= n)
                        w.batch.bad();
                    at = entry < n ? entry : -1;
                    key0 = at * w.cache.page + (key & (w.cache.page - 1));
                }
                if (at >= 0 && key0 < ctx) {
                    p = w.batch.page(b, at);
                    if (p < 0)
                        w.batch.bad();
                }
            }
            const int ph = p * w.cache.heads + head;
            if (p >= 0) {
                ks = w.cache.k_scale[ph];
                vs = w.cache.v_scale[ph];
            }
            const unsigned alive = __ballot_sync(0xffffffffu, p >= 0);
            // lane l < SUBS writes the record of a stage's tile l: the lane that has its copy
            const int tile_lane = (lane * kTile) >> w.log2_box, tile_key = (lane * kTile) & (box - 1);
            for (int u = 0; u < here; ++u, ++done) {
                if (done >= S && !(ok = wait_warp(empty(s), phase ^ 1u, abort_flag)))
                    break;
                const int first_lane = u << log2_boxes;
                const bool mine = (lane >> log2_boxes) == u;
                const bool ended = unit + 1 == units || done + 1 == all;
                // the copies first (their bytes may arrive before they are
                // expected: the phase waits for the arrival below), then the
                // record, whose scales may still be under way
                if (mine && p >= 0) {
                    const int row0 = (lane - first_lane) << w.log2_box;  // of the stage
                    const uint32_t dst = sbase + F::RING_OFF + s * F::STAGE + row0 * F::W0;
                    const int y = key0 & (w.cache.page - 1);
                    tma_load_3d(dst, &maps.k[0], full(s), 0, y, ph, policy, box * F::W0);
                    tma_load_3d(dst + F::HALF, &maps.v[0], full(s), 0, y, ph, policy, box * F::W0);
                    if (F::PARTS == 2) {
                        const uint32_t dst1 = sbase + F::RING_OFF + s * F::STAGE + F::STEP * F::W0 + row0 * F::W1;
                        tma_load_3d(dst1, &maps.k[1], full(s), F::W0, y, ph, policy, box * F::W1);
                        tma_load_3d(dst1 + F::HALF, &maps.v[1], full(s), F::W0, y, ph, policy, box * F::W1);
                    }
                }
                StageMeta *m = meta + s;
                const int from = (first_lane + tile_lane) & 31;
                const float tk = __shfl_sync(0xffffffffu, ks, from), tv = __shfl_sync(0xffffffffu, vs, from);
                const int t0 = __shfl_sync(0xffffffffu, key0, from) + tile_key;
                const int v_exp = static_cast<int>(__float_as_uint(tv) >> 23);
                const float v_inv = __int_as_float((254 - v_exp) << 23);
                const bool odd = lane < F::SUBS && tv * v_inv != 1.f;
                if (lane < F::SUBS) {
                    const bool seen = (alive >> from & 1u) && t0 < ctx;
                    m->tile[lane] = {tk, static_cast<float>(v_exp - 127), v_inv, seen ? t0 : kNoKey};
                }
                int flags = (opened ? kFirst : 0) | (ended ? kLast : 0) | (__any_sync(0xffffffffu, odd) ? kOddScale : 0);
                if (ended) {
                    // did this block have the segment from its first to its last unit?
                    if (unit > done)
                        flags |= kHeadPart;  // it began before this block's run
                    else if (unit + 1 < units)
                        flags |= kTailPart;
                }
                if ((flags & kOddScale) && lane < F::SUBS)
                    m->v_rest[lane] = tv * v_inv;
                if (lane == 0) {
                    m->flags = flags;
                    if (opened) {
                        m->b = b;
                        m->i = i;
                        m->head = head;
                        m->group = group;
                    }
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_expect_tx(full(s), __popc(alive >> first_lane & stage_lanes) * 2 * box * D);
                opened = ended;
                ++unit;
                if (++s == S) {
                    s = 0;
                    phase ^= 1u;
                }
            }
            if (unit == units && done < all) {  // on to the next segment
                unit = 0;
                if (++group == w.groups) {
                    group = 0;
                    if (++head == w.cache.heads) {
                        head = 0;
                        do {
                            if (++i >= (w.pages ? w.q.Nq : 1)) {
                                i = 0;
                                ++b;
                            }
                            open_query();
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
    const int key_warps = kDecWarps / w.row_warps;
    const int wk = warp % key_warps, wr = warp / key_warps;
    // Q^T operand: of query rows g (+ 8), their d in the order of the thread's K
    // words; in registers for eight rows, for sixteen in the warp's merge area
    // (each lane its own), where registers would cost a third of the warps
    uint32_t qb[NT == 1 ? KW : 1][2];
    const uint32_t q_own = sbase + F::MERGE_OFF + warp * (8 * F::OROW * 4) + lane * 16;
    static_assert(KW * 512 <= 8 * F::OROW * 4, "sixteen rows of Q fit the merge area");
    float qf[NT][2];          // per query row 2 c, 2 c + 1 (+ 8): scale to log2 units
    uint32_t behind = 0;      // ... keys that it sees beyond `least`, a byte each
    float m[NT][2], l[NT][2], acc[D / 16][NT][4];
    int least = 0, most = 0;  // keys that all rows see (negative: the first ones see none), that any row sees
    auto limit = [&](int nt, int u) -> int { return least + static_cast<int>((behind >> (8 * (2 * nt + u))) & 255u); };
    int4 *segment = reinterpret_cast<int4 *>(smem + F::FLAG_OFF + 16) + warp;  // b, i, head, group
    uint32_t merges = 0;
    // a barrier of the computing warps whose wait is bounded
    auto meet = [&]() -> bool {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(merged);
        return wait_warp(merged, merges++ & 1u, abort_flag);
    };
    bool fresh = true;   // some row may have no reference yet
    uint32_t unset = 0;  // ... a bit each of the thread's
    int slot = S - 1;
    uint32_t phase = 1;
    for (int done = 0; done < all; ++done) {
        if (++slot == S)
            slot = 0;
        if (slot == 0)
            phase ^= 1u;
        if (!wait_warp(full(slot), phase, abort_flag))
            return;
        const StageMeta *info = meta + slot;
        const int flags = info->flags;
        const bool odd_scale = flags & kOddScale;  // a V scale that is no power of two

        if (flags & kFirst) {
            const int b_seg = info->b, i_seg = info->i;
            head = info->head;
            group = info->group;
            if (lane == 0)
                *segment = make_int4(b_seg, i_seg, head, group);
            __syncwarp();
            const int n = w.batch.length(b_seg, w.cache.log2_page);
            most = w.pages ? context(w.q, n, i_seg) : n;
            least = w.pages || !w.q.causal ? most : n - w.q.Nq + 1;
            behind = 0;
            fresh = true;
            unset = (1u << (2 * NT)) - 1u;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int row = group * rows_block + wr * ROWS + nt * 8 + g;
                const int hq = w.pages ? row : row / w.q.Nq, qi = w.pages ? i_seg : row % w.q.Nq;
                const T *src = static_cast<const T *>(w.q.q) + b_seg * w.q.batch_stride +
                               static_cast<long long>(head * w.q.G + hq) * w.q.head_stride + qi * w.q.row_stride;
                uint2 x[KW];
                float top = 0.f;
#pragma unroll
                for (int s = 0; s < KW; ++s) {
                    x[s] = make_uint2(0, 0);
                    if (row < w.R)
                        x[s] = *reinterpret_cast<const uint2 *>(src + k_column<D>(c, s));
                }
#pragma unroll
                for (int s = 0; s < KW; ++s) {
                    const float2 y = DTypeTraits<T>::unpack(x[s].x), z = DTypeTraits<T>::unpack(x[s].y);
                    const float f[4] = {fabsf(y.x), fabsf(y.y), fabsf(z.x), fabsf(z.y)};
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (f[u] <= 3.402823466e38f)
                            top = fmaxf(top, f[u]);
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = top > 0.f ? max(static_cast<int>(__float_as_uint(top) >> 23) - 127 - 14, -100) : 0;
                const float by = pow2f(-e);
#pragma unroll
                for (int s = 0; s < KW; ++s) {
                    const float2 y = DTypeTraits<T>::unpack(x[s].x), z = DTypeTraits<T>::unpack(x[s].y);
                    const uint32_t b0 = DTypeTraits<__half>::pack(y.x * by, y.y * by);
                    const uint32_t b1 = DTypeTraits<__half>::pack(z.x * by, z.y * by);
                    if constexpr (NT == 1) {
                        qb[s][0] = b0;
                        qb[s][1] = b1;
                    } else {
                        store_pair(q_own + s * 512 + nt * 8, b0, b1);
                    }
                }
                const int extra = w.pages || !w.q.causal ? 0 : qi;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    qf[nt][u] = pow2f(__shfl_sync(0xffffffffu, e, 8 * c + 4 * u)) * w.scale_log2;
                    behind |= __shfl_sync(0xffffffffu, extra, 8 * c + 4 * u) << (8 * (2 * nt + u));
                    m[nt][u] = 0.f;
                    l[nt][u] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        acc[j][nt][u] = 0.f;
            }
        }

        for (int set = wk; set < F::SUBS / J; set += key_warps) {
            // J tiles at once: one look at the reference, and twice the independent work
            const int sub0 = set * J;
            const bool last_set = set + key_warps >= F::SUBS / J;
            TileMeta tile[J];
            int key0[J];
            int nearest = kNoKey, farthest = 0;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                tile[j] = info->tile[sub0 + j];
                key0[j] = tile[j].key0;
                nearest = min(nearest, key0[j]);
                farthest = max(farthest, key0[j]);
            }
            if (nearest == kNoKey) {
                if (last_set) {
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(empty(slot));
                }
                continue;
            }
            const uint32_t k0 = sbase + F::RING_OFF + slot * F::STAGE + sub0 * kTile * F::W0, v0 = k0 + F::HALF;
            const uint32_t k1 = sbase + F::RING_OFF + slot * F::STAGE + F::STEP * F::W0 + sub0 * kTile * F::W1;  // d = 96
            // ---- S^T = K Q^T ----
            float e[J][NT][4];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                uint32_t kw[2][KW];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t kj = k0 + j * kTile * F::W0;
                    if constexpr (D == 128) {
                        load_words<4>(&kw[r][0], kj + k_offset<128>(g, c, 0) + r * 1024);
                        load_words<4>(&kw[r][4], kj + k_offset<128>(g, c, 1) + r * 1024);
                    } else if constexpr (D == 32) {
                        load_words<2>(&kw[r][0], kj + k_offset<32>(g, c, 0) + r * 256);
                    } else {
                        load_words<4>(&kw[r][0], kj + k_offset<64>(g, c, 0) + r * 512);
                    }
                    if constexpr (D == 96)
                        load_words<2>(&kw[r][4], k1 + j * kTile * F::W1 + k_offset<32>(g, c, 0) + r * 256);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        e[j][nt][u] = 0.f;
#pragma unroll
                for (int x = 0; x < KW; ++x) {
                    uint32_t a0, a1, a2, a3;
                    C::halves(kw[0][x], a0, a2);
                    C::halves(kw[1][x], a1, a3);
                    if constexpr (NT == 1) {
                        mma_f16(e[j][0], a0, a1, a2, a3, qb[x][0], qb[x][1]);
                    } else {
                        uint32_t y[4];
                        load_words<4>(y, q_own + x * 512);
                        mma_f16(e[j][0], a0, a1, a2, a3, y[0], y[1]);
                        mma_f16(e[j][1], a0, a1, a2, a3, y[2], y[3]);
                    }
                }
            }
            // ---- exponents of P v_scale, masks; does any outgrow its reference? ----
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        e[j][nt][u] = fmaf(e[j][nt][u], tile[j].k_scale * qf[nt][u & 1], tile[j].v_log2 - m[nt][u & 1]);
            const bool masked = farthest + kTile > least;
            if (masked) {
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            if (key0[j] + g + 8 * (u >> 1) >= limit(nt, u & 1))
                                e[j][nt][u] = -INFINITY;
            }
            bool grown = fresh;
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        grown |= !(e[j][nt][u] <= kMost);
            if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint32_t bit = 1u << (2 * nt + u);
                        float top = -INFINITY;  // over the reference, which is 0 as long as it is not set
#pragma unroll
                        for (int j = 0; j < J; ++j)
                            top = fmaxf(top, fmaxf(e[j][nt][u], e[j][nt][u + 2]));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                        const float over = top - kAim;
                        const float up = unset & bit ? (top == -INFINITY ? 0.f : over) : fmaxf(over, 0.f);
                        const float alpha = unset & bit ? 1.f : ex2(-up);
                        if (top > -INFINITY)
                            unset &= ~bit;
                        m[nt][u] += up;
                        l[nt][u] *= alpha;
#pragma unroll
                        for (int j = 0; j < J; ++j) {
                            e[j][nt][u] -= up;
                            e[j][nt][u + 2] -= up;
                        }
#pragma unroll
                        for (int j = 0; j < D / 16; ++j) {
                            acc[j][nt][u] *= alpha;
                            acc[j][nt][u + 2] *= alpha;
                        }
                    }
                fresh = __any_sync(0xffffffffu, unset != 0);
            }
            // ---- P, and O^T += V^T P^T ----
            uint32_t pb[J][NT][2];
#pragma unroll
            for (int j = 0; j < J; ++j) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float(&p)[4] = e[j][nt];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        p[u] = ex2(p[u]);
                        l[nt][u & 1] = fmaf(p[u], tile[j].v_inv, l[nt][u & 1]);
                    }
                    if (odd_scale) {
                        const float rest = info->v_rest[sub0 + j];
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            p[u] *= rest;
                    }
                    pb[j][nt][0] = transpose8(DTypeTraits<__half>::pack(p[0], p[1]));
                    pb[j][nt][1] = transpose8(DTypeTraits<__half>::pack(p[2], p[3]));
                }
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const uint32_t vj = v0 + j * kTile * F::W0;
                uint32_t vw[4][VW];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if constexpr (D == 128)
                        load_words<4>(&vw[r][0], vj + v_offset<128>(g, c, r & 1) + (r >> 1) * 1024);
                    else if constexpr (D == 32)
                        load_words<1>(&vw[r][0], vj + v_offset<32>(g, c, r & 1) + (r >> 1) * 256);
                    else
                        load_words<2>(&vw[r][0], vj + v_offset<64>(g, c, r & 1) + (r >> 1) * 512);
                    if constexpr (D == 96)
                        load_words<1>(&vw[r][2],
                                      k1 + j * kTile * F::W1 + F::HALF + v_offset<32>(g, c, r & 1) + (r >> 1) * 256);
                }
                if (j == J - 1 && last_set) {  // the stage's codes are in registers
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(empty(slot));
                }
                if (masked) {
                    // codes behind the last key are whatever the page held
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (key0[j] + 2 * c + (r & 1) + 8 * (r >> 1) >= most)
#pragma unroll
                            for (int x = 0; x < VW; ++x)
                                vw[r][x] = 0;
                    if (C::kUnit != 1) {
                        // NaN codes of V at keys that some rows do not see: 0 * NaN
                        // must not reach those rows, so the rows that do see such a
                        // key get their NaN here and the code becomes 0
                        uint32_t any = 0;
#pragma unroll
                        for (int r = 0; r < 4; ++r)
#pragma unroll
                            for (int x = 0; x < VW; ++x)
                                any |= nan_bytes(vw[r][x]);
                        if (__any_sync(0xffffffffu, any != 0)) {
#pragma unroll 1
                            for (int key = 0; key < kTile; ++key) {
                                const int r = (key & 1) + 2 * (key >> 3), from = (lane & ~3) | ((key & 7) >> 1);
#pragma unroll
                                for (int x = 0; x < VW; ++x) {
                                    const uint32_t own =
                                        r == 0 ? vw[0][x] : r == 1 ? vw[1][x] : r == 2 ? vw[2][x] : vw[3][x];
                                    const uint32_t bits = nan_bytes(__shfl_sync(0xffffffffu, own, from));
#pragma unroll
                                    for (int y = 0; y < 4; ++y)
#pragma unroll
                                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                            for (int u = 0; u < 2; ++u)
                                                if ((bits >> (8 * y + 7) & 1u) && key0[j] + key < limit(nt, u))
                                                    acc[2 * x + (y >> 1)][nt][(y & 1) * 2 + u] = __int_as_float(0x7FC00000);
                                }
                            }
#pragma unroll
                            for (int r = 0; r < 4; ++r)
#pragma unroll
                                for (int x = 0; x < VW; ++x) {
                                    const uint32_t bits = nan_bytes(vw[r][x]);
                                    vw[r][x] &= ~((bits >> 7) * 0xFFu);
                                }
                        }
                    }
                }
#pragma unroll
                for (int x = 0; x < VW; ++x) {
                    // four columns of V: bytes of keys 2 c, 2 c + 1 and 2 c + 8, 2 c + 9 side by side
                    uint32_t a[4][2];  // column, key pair
                    C::halves(__byte_perm(vw[0][x], vw[1][x], 0x5140), a[0][0], a[1][0]);
                    C::halves(__byte_perm(vw[0][x], vw[1][x], 0x7362), a[2][0], a[3][0]);
                    C::halves(__byte_perm(vw[2][x], vw[3][x], 0x5140), a[0][1], a[1][1]);
                    C::halves(__byte_perm(vw[2][x], vw[3][x], 0x7362), a[2][1], a[3][1]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_f16(acc[2 * x][nt], a[0][0], a[1][0], a[0][1], a[1][1], pb[j][nt][0], pb[j][nt][1]);
                        mma_f16(acc[2 * x + 1][nt], a[2][0], a[3][0], a[2][1], a[3][1], pb[j][nt][0], pb[j][nt][1]);
                    }
                }
            }
        }

        if (flags & kLast) {
            // ---- merge the warps of each row group, eight rows a warp at a time;
            // write the rows, or the block's part ----
            float *mo = reinterpret_cast<float *>(smem + F::MERGE_OFF);
            float *mm = reinterpret_cast<float *>(smem + F::ML_OFF), *ml = mm + kDecWarps * 8;
            const int b_seg = segment->x, i_seg = segment->y;
            head = segment->z;
            group = segment->w;
            const bool part = flags & (kHeadPart | kTailPart);
            const long long place = 2ll * blockIdx.x + (flags & kTailPart ? 1 : 0);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float sum = l[nt][u];
                    sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                    const int row = warp * 8 + 2 * c + u;
                    if (g == 0) {
                        mm[row] = unset >> (2 * nt + u) & 1u ? -INFINITY : m[nt][u];
                        ml[row] = sum;
                    }
#pragma unroll
                    for (int x = 0; x < VW; ++x)
                        *reinterpret_cast<float4 *>(mo + row * F::OROW + v_column<D>(g, x)) =
                            make_float4(acc[2 * x][nt][u], acc[2 * x][nt][u + 2], acc[2 * x + 1][nt][u],
                                        acc[2 * x + 1][nt][u + 2]);
                }
                if (!meet())
                    return;
                for (int x = t; x < 8 * w.row_warps * (D / 2); x += 32 * kDecWarps) {
                    const int r8 = x / (D / 2), d = 2 * (x % (D / 2));
                    const int row = r8 / 8 * ROWS + nt * 8 + r8 % 8;  // of the block
                    const int abs_row = group * rows_block + row;
                    if (abs_row >= w.R)
                        continue;
                    const int from = (r8 / 8) * key_warps * 8 + r8 % 8;  // of its first warp
                    float top = -INFINITY;
                    for (int y = 0; y < key_warps; ++y)
                        top = fmaxf(top, mm[from + y * 8]);
                    float2 o = make_float2(0.f, 0.f);
                    float sum = 0.f;
                    const float ref = top == -INFINITY ? 0.f : top;
                    for (int y = 0; y < key_warps; ++y) {
                        const float f = ex2(mm[from + y * 8] - ref);
                        const float2 z = *reinterpret_cast<const float2 *>(mo + (from + y * 8) * F::OROW + d);
                        o.x = fmaf(z.x, f, o.x);
                        o.y = fmaf(z.y, f, o.y);
                        sum = fmaf(ml[from + y * 8], f, sum);
                    }
                    if (part) {
                        const long long pr = place * rows_block + row;
                        *reinterpret_cast<float2 *>(w.part_o + pr * D + d) = o;
                        if (d == 0) {
                            w.part_m[pr] = top;
                            w.part_l[pr] = sum;
                        }
                    } else {
                        const long long bh = static_cast<long long>(b_seg) * w.cache.heads + head;
                        const long long orow = w.pages ? (bh * w.q.G + abs_row) * w.q.Nq + i_seg : bh * w.R + abs_row;
                        const float inv = sum == 0.f ? 0.f : 1.f / sum;
                        *reinterpret_cast<uint32_t *>(out + orow * D + d) = DTypeTraits<T>::pack(o.x * inv, o.y * inv);
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

// Merges the parts of every segment that more than one block has, SPLIT warps a
// query row; writes the rows of segments without keys.  Units are of 2^LOG2_STEP keys, and
// the first of a segment lies OPEN behind its begin.
template <int D, typename T, int SPLIT, int LOG2_STEP = DecCfg<D>::LOG2_STEP, int OPEN = 0>
__global__ void __launch_bounds__(kCombineThreads)
    fa_cache_combine_kernel(const __grid_constant__ Work w, T *__restrict__ out, float *__restrict__ lse, int rows_block,
                            long long rows)
{
    constexpr int WARPS = kCombineThreads / 32;
    __shared__ __align__(16) float red_o[SPLIT > 1 ? WARPS : 1][D];
    __shared__ float red_m[WARPS], red_l[WARPS];
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % SPLIT;
    // row = ((b * queries + i) * heads + head) * R + row of the segment
    const int queries = w.pages ? w.q.Nq : 1;
    long long x = static_cast<long long>(blockIdx.x) * (WARPS / SPLIT) + (threadIdx.x >> 5) / SPLIT;
    if (x >= rows)
        return;
    const int row = static_cast<int>(x % w.R);
    x /= w.R;
    const int head = static_cast<int>(x % w.cache.heads);
    x /= w.cache.heads;
    const int i = static_cast<int>(x % queries), b = static_cast<int>(x / queries);
    const int group = row / rows_block;
    const int len = w.batch.length(b, w.cache.log2_page);
    const int units = units_of<LOG2_STEP>(w, len, i);
    const long long orow =
        w.pages ? ((static_cast<long long>(b) * w.cache.heads + head) * w.q.G + row) * w.q.Nq + i
                : (static_cast<long long>(b) * w.cache.heads + head) * w.R + row;
    if (units == 0) {
        wait_ahead();
        for (int d = 2 * (32 * warp + lane); d < D; d += 64 * SPLIT)
            *reinterpret_cast<uint32_t *>(out + orow * D + d) = 0;
        if (lane == 0 && warp == 0 && lse != nullptr)
            lse[orow] = -INFINITY;
        return;
    }
    wait_ahead();
    const long long share = w.plan[0];
    long long first = w.plan[1 + b];
    for (int y = 0; y < i; ++y) {
        const int n = units_of<LOG2_STEP>(w, len, y);
        first += static_cast<long long>(n > 0 ? n + OPEN : 0) * w.cache.heads * w.groups;
    }
    first += (static_cast<long long>(head) * w.groups + group) * (units + OPEN) + OPEN;
    const int x0 = static_cast<int>(first / share), x1 = static_cast<int>((first + units - 1) / share);
    if (x0 == x1)
        return;  // one block had it all, and has written it
    const int in_block = row % rows_block;
    // warp v: the parts of blocks x0 + v, + SPLIT, ..., several at once; lane: columns 4 lane .. 4 lane + 3
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float top = -INFINITY, sum = 0.f;
    for (int y0 = x0 + warp; y0 <= x1; y0 += SPLIT * kCombineEach) {
        float m[kCombineEach], l[kCombineEach];
        float4 z[kCombineEach];
#pragma unroll
        for (int u = 0; u < kCombineEach; ++u) {
            const int y = y0 + u * SPLIT;
            m[u] = -INFINITY;
            l[u] = 0.f;
            z[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (y <= x1) {
                // a block's place: its head part if the segment began before its run
                const long long p = (2ll * y + (y * share > first ? 0 : 1)) * rows_block + in_block;
                m[u] = w.part_m[p];
                l[u] = w.part_l[p];
                if (4 * lane < D)
                    z[u] = *reinterpret_cast<const float4 *>(w.part_o + p * D + 4 * lane);
            }
        }
        float next = top;
#pragma unroll
        for (int u = 0; u < kCombineEach; ++u)
            next = fmaxf(next, m[u]);
        // no key so far, or only NaN scores, whose sum is NaN: factors of 0
        const float ref = next == -INFINITY ? 0.f : next;
        const float alpha = ex2(top - ref);
        top = next;
        sum *= alpha;
        o = make_float4(o.x * alpha, o.y * alpha, o.z * alpha, o.w * alpha);
#pragma unroll
        for (int u = 0; u < kCombineEach; ++u) {
            const float f = ex2(m[u] - ref);
            sum = fmaf(l[u], f, sum);
            o.x = fmaf(z[u].x, f, o.x);
            o.y = fmaf(z[u].y, f, o.y);
            o.z = fmaf(z[u].z, f, o.z);
            o.w = fmaf(z[u].w, f, o.w);
        }
    }
    if (SPLIT > 1) {  // a block has one row: join its warps
        if (4 * lane < D)
            *reinterpret_cast<float4 *>(&red_o[warp][4 * lane]) = o;
        if (lane == 0) {
            red_m[warp] = top;
            red_l[warp] = sum;
        }
        __syncthreads();
        if (warp != 0)
            return;
        top = red_m[0];
#pragma unroll
        for (int y = 1; y < SPLIT; ++y)
            top = fmaxf(top, red_m[y]);
        sum = 0.f;
        o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int y = 0; y < SPLIT; ++y) {
            const float f = red_m[y] == -INFINITY ? 0.f : ex2(red_m[y] - top);
            sum = fmaf(red_l[y], f, sum);
            if (4 * lane < D) {
                const float4 z = *reinterpret_cast<const float4 *>(&red_o[y][4 * lane]);
                o.x = fmaf(z.x, f, o.x);
                o.y = fmaf(z.y, f, o.y);
                o.z = fmaf(z.z, f, o.z);
                o.w = fmaf(z.w, f, o.w);
            }
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (4 * lane < D)
        *reinterpret_cast<uint2 *>(out + orow * D + 4 * lane) =
            make_uint2(DTypeTraits<T>::pack(o.x * inv, o.y * inv), DTypeTraits<T>::pack(o.z * inv, o.w * inv));
    if (lane == 0 && lse != nullptr)
        lse[orow] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * 0.6931471805599453f;
}

}  // namespace cache
}  // namespace fa
