// fa_cache4_tc_kernel.cuh -- decoding attention over the 4-bit paged cache for more than 32 query
// rows a KV head, at d = 128 more than 16, with the products on tcgen05 (but batches of short
// segments: on_tcgen05 in fa_cache4.cu, with both sides' figures).
//
// The kernel of fa_cache4_decode_kernel.cuh converts a tile's codes in registers, once for every
// 16 rows.  Here they are converted once for the 32 or 64 rows of a group, into fp16 tiles of K and V
// in shared memory, swizzled as the tensor cores read them:
//   S^T = K Q^T     M = 128 keys, N = rows, K = d; K and Q K-major
//   O^T += V^T P^T  M = 128 (d, the columns of V behind it zero), N = rows, K = 128 keys; V read
//                   MN-major, and so is P^T, a row of it a key
// with fp32 accumulators in TMEM, S^T in two buffers.  Runs, ring, records, parts and their merge
// are those of the other kernel; so is the softmax (P in fp16, 2^kAim under the largest weight, a
// reference that moves only when one outgrows it).
//
// Warps: eight or sixteen do the softmax, four for every 16 rows (a thread has a key of S^T, a channel of
// O^T, and their 16 rows), four convert K and four V, one copies, two issue the products.  K and
// V of a unit are apart: K's tile is free when its product is done, V's only when the one with
// P^T is, and with eight warps for both one after the other a unit took a tenth longer.
//
// What bounds it: the chain of a unit.  Converting, product, softmax, product take some 6,000
// clocks, and two units under way make about 2,900 each (64 rows), in which 1,700 instructions of a
// scheduler issue; HBM would need 800, shared memory, through which every converted byte goes
// twice, 1,000.  The softmax alone (S^T from TMEM, a barrier of four warps for the references,
// P^T back) is 1,700.
//
// Measured on the GPU, 8 KV heads, this kernel / the other, us.  16 sequences of up to 16,384 keys;
// one of 60,000; 64 of 2,000; 100 of 700; one of 500; 8 of 100:
//   d = 128, 64 rows  110 / 182  49 / 80  87 / 115  83 / 99  14 / 21  10 / 12
//            36       105 / 179  47 / 79  79 / 106  74 / 86  14 / 19  10 / 10
//            32        84 / 98   38 / 48  63 / 66   58 / 58  11 / 13   8.0 / 8.6
//            18        82 / 97   37 / 46  58 / 60   54 / 51  11 / 12   8.0 / 7.7
//   d = 96,  64       107 / 156  47 / 66  85 / 99   83 / 83  14 / 18  10 / 10
//            36       102 / 153  45 / 65  78 / 90   73 / 71  13 / 17  10 / 9
//            32 (not taken) 84 / 87, 38 / 41, 63 / 57, 59 / 50, 11 / 11, 8.0 / 7.4
//   d = 64,  64 (not taken) 99 / 110, 43 / 49, 92 / 75, 86 / 65, 13 / 14, 9 / 8
// Of the first case: two tiles of P^T and two stages 116, one tile of P^T at d = 96 116; OPEN of 2 120,
// of 6 118 where 4 took 116; four warps that convert 121, sixteen (32 rows) 93.
#pragma once

#include "fa_cache4_run.cuh"
#include "fa_cache4_running.cuh"

namespace fa {
namespace cache4 {

template <int D, int ROWS_>
struct Tc4Cfg {
    static_assert((D == 96 && ROWS_ == 64) || (D == 128 && (ROWS_ == 32 || ROWS_ == 64)), "what the launch chooses");
    static constexpr int D_ = D;
    static constexpr int ROWS = ROWS_;  // of a group
    static constexpr int LOG2_STEP = 7;
    static constexpr int STEP = 1 << LOG2_STEP;
    static constexpr int STAGE = STEP * D / 8 * 9;
    static constexpr int OPEN = 4;  // units that a segment's begin and end cost
    static constexpr int SOFTMAX = ROWS / 4, CONVERT = 8;  // warps
    static constexpr int LOAD_WARP = SOFTMAX + CONVERT, S_WARP = LOAD_WARP + 1, O_WARP = S_WARP + 1;
    static constexpr int THREADS = 32 * (O_WARP + 1);
    static constexpr int STAGES = 3;
    static constexpr int PS = D == 128 && ROWS == 64 ? 1 : 2;  // tiles of P^T: a stage is worth more than a second one
    static constexpr int KTILE = 2 * kSwAtomBytes;  // K or V of a unit: two 64-column blocks of 128-byte rows
    static constexpr int TILE = 2 * KTILE;          // two of them
    static constexpr int BLK = ROWS * 128;      // a 64-column block of Q
    static constexpr int QTILE = 2 * BLK, PTILE = kSwAtomBytes;  // of P^T a 128-byte row a key
    static constexpr int Q_OFF = 2 * TILE;
    static constexpr int P_OFF = Q_OFF + QTILE;
    static constexpr int RING_OFF = P_OFF + PS * PTILE;
    static constexpr int META_OFF = RING_OFF + STAGES * STAGE;  // records of stages, and of four units each of K and V
    static constexpr int ROW_OFF = META_OFF + (STAGES + 8) * 32;  // of each row: scale, reference, last key, factor
    static constexpr int RED_OFF = ROW_OFF + 4 * ROWS * 4;        // [4 warps][ROWS]
    static constexpr int BAR_OFF = RED_OFF + 4 * ROWS * 4;
    static constexpr int B_EMPTY = STAGES;       // of the ring, behind the full ones
    static constexpr int B_KFULL = 2 * STAGES;   // 2: a unit's K is converted
    static constexpr int B_VFULL = B_KFULL + 2;  // 2
    static constexpr int B_SFULL = B_VFULL + 2;  // 2: S^T is there
    static constexpr int B_SFREE = B_SFULL + 2;  // 2: ... and read
    static constexpr int B_PFULL = B_SFREE + 2;  // 2: P^T is written
    static constexpr int B_ODONE = B_PFULL + 2;  // 2: the products with a tile are done
    static constexpr int B_QFULL = B_ODONE + 2;
    static constexpr int B_OFREE = B_QFULL + 1;  // O^T is read
    static constexpr int B_DRAIN = B_OFREE + 1;  // 2
    static constexpr int BARS = B_DRAIN + 2;
    static constexpr int SLOT_OFF = BAR_OFF + 8 * BARS;  // TMEM address, abort flag
    static constexpr int SMEM = SLOT_OFF + 16 + 1024;    // and room to align the tiles
    static constexpr uint32_t TM_O = 2 * ROWS, TM_COLS = ROWS == 64 ? 256 : 128;
    static_assert(SMEM <= 227 * 1024 && RING_OFF % 1024 == 0 && STAGE % 128 == 0, "shared memory");
};

template <typename T>
__device__ __forceinline__ T to_type(float x);
template <>
__device__ __forceinline__ __half to_type<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 to_type<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Byte offset of element (row, col) of a tile of 128-byte rows in 64-column blocks of BLK bytes, swizzled.
template <int BLK>
__device__ __forceinline__ uint32_t tile_offset(int row, int col)
{
    return static_cast<uint32_t>((col >> 6) * BLK + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4) + (col & 7) * 2);
}

template <int D, int ROWS_, typename T>
__global__ void __launch_bounds__(Tc4Cfg<D, ROWS_>::THREADS, 1)
    fa_cache4_tc_kernel(const __grid_constant__ Work w, T *__restrict__ out, float *__restrict__ lse)
{
    using F = Tc4Cfg<D, ROWS_>;
    constexpr int S = F::STAGES, ROWS = F::ROWS;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (sbase - raw);
    auto bar = [&](int x) -> uint32_t { return sbase + F::BAR_OFF + 8u * x; };
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + F::SLOT_OFF);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + F::SLOT_OFF + 4);
    Stage4 *meta = reinterpret_cast<Stage4 *>(smem + F::META_OFF), *of_k = meta + S, *of_v = of_k + 4;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;

    if (t == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(bar(s), 1);
            mbar_init(bar(F::B_EMPTY + s), F::CONVERT);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(F::B_KFULL + i), F::CONVERT / 2);
            mbar_init(bar(F::B_VFULL + i), F::CONVERT / 2);
            mbar_init(bar(F::B_SFULL + i), 1);
            mbar_init(bar(F::B_SFREE + i), F::SOFTMAX);
            mbar_init(bar(F::B_PFULL + i), F::SOFTMAX);
            mbar_init(bar(F::B_ODONE + i), 1);
            mbar_init(bar(F::B_DRAIN + i), 1);
        }
        mbar_init(bar(F::B_QFULL), F::SOFTMAX);
        mbar_init(bar(F::B_OFREE), F::SOFTMAX);
        *abort_flag = 0;
        fence_mbar_init();
    }
    cache::wait_ahead();
    cache::let_next();
    Run run;
    if (!find_run<F>(w, run))
        return;
    if (warp == F::S_WARP) {
        tmem_alloc(smem_u32(const_cast<uint32_t *>(tmem_slot)), F::TM_COLS);
        tmem_relinquish();
    }
    if (D < 128 && warp < F::SOFTMAX) {  // V's columns behind d, which no unit writes
        for (int x = t; x < 2 * (F::KTILE / 16); x += 32 * F::SOFTMAX)
            st_shared_v4(sbase + x / (F::KTILE / 16) * F::TILE + F::KTILE + x % (F::KTILE / 16) * 16, 0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int log2_page = w.cache.log2_page;
    const int box = 1 << w.log2_box, box_bytes = box * (D / 8 * 9);
    const unsigned all_boxes = (1u << (F::STEP >> w.log2_box)) - 1u;

    if (warp == F::LOAD_WARP) {
        load_run<F>(w, run, sbase + F::RING_OFF, meta, bar(0), abort_flag);
    } else if (warp >= F::SOFTMAX && warp < F::LOAD_WARP) {
        // ---------------- the warps that convert ----------------
        constexpr int THREADS = 16 * F::CONVERT;  // half for K, half for V
        const bool is_v = t - 32 * F::SOFTMAX >= THREADS;
        const int x = (t - 32 * F::SOFTMAX) % THREADS;
        constexpr int PIECES = D / 32;  // of a row of codes, 16 bytes each
        int len = 0;
        for (int i = 0, flags = 0; !(flags & kEnd); ++i) {
            const int s = i % S, buf = i & 1;
            if (!wait_warp(bar(s), (i / S) & 1, abort_flag))
                break;
            const int4 info = *reinterpret_cast<const int4 *>(meta + s);  // flags, unit, b, head
            flags = info.x;
            if (flags & kFirst)
                len = w.batch.length(info.z, log2_page);
            // K's tile is free when its product is done, V's when the one with P^T is
            if (i >= 2 && !wait_warp(bar((is_v ? F::B_ODONE : F::B_SFULL) + buf), ((i >> 1) - 1) & 1, abort_flag))
                break;
            if (x < 2)
                reinterpret_cast<int4 *>((is_v ? of_v : of_k) + (i & 3))[x] = reinterpret_cast<const int4 *>(meta + s)[x];
            const uint32_t from = sbase + F::RING_OFF + s * F::STAGE + (is_v ? box_bytes / 2 : 0);
            const uint32_t to = sbase + buf * F::TILE + (is_v ? F::KTILE : 0);
            const int seen = min(len - (info.y << F::LOG2_STEP), F::STEP);  // keys of this unit
#pragma unroll 4
            for (int id = x; id < 128 * PIECES; id += THREADS) {
                const int row = id / PIECES, c = id % PIECES, in_box = row & (box - 1), number = row >> w.log2_box;
                const uint32_t at = from + number * box_bytes;
                uint32_t v[4];
                cache::load_words<4>(v, at + in_box * (D / 2) + c * 16);
                uint32_t by = load_u16(at + box * (D / 2) + in_box * (D / 16) + 2 * c);
                // what lies behind the last key, or was not copied, may hold scales that are none: S^T is
                // masked, V has to be finite
                if (!(flags >> (kBoxes + number) & 1) || row >= seen)
                    by = 0;
                // eight channels a store; where four pieces make a row the order of a lane's stores keeps eight
                // lanes, two rows, apart in the banks
                int turn = row & 7;
                if constexpr (PIECES == 4) {
                    const bool a = c & 2, z = row & 1;
                    turn ^= (a ? 1 : 0) | (z ? 2 : 0);
                    uint32_t y[4] = {a ? v[1] : v[0], a ? v[0] : v[1], a ? v[3] : v[2], a ? v[2] : v[3]};
                    v[0] = z ? y[2] : y[0], v[1] = z ? y[3] : y[1], v[2] = z ? y[0] : y[2], v[3] = z ? y[1] : y[3];
                    by = z ? by >> 8 | (by & 255u) << 8 : by;
                }
                turn ^= (c & 1) * 4;
                const uint32_t dst = to + (c >> 1) * kSwAtomBytes + row * 128;
                const uint32_t scales[2] = {(by & 255u) * 0x800080u, (by >> 8) * 0x800080u};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint32_t h[4];
                    halves8(v[u], h);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        h[j] = times(h[j], scales[u >> 1]);
                    st_shared_v4(dst + ((turn ^ u) << 4), h[0], h[1], h[2], h[3]);
                }
            }
            fence_proxy_async_smem();  // read by the tensor cores
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar((is_v ? F::B_VFULL : F::B_KFULL) + buf));
                mbar_arrive(bar(F::B_EMPTY + s));
            }
        }
    } else if (warp == F::S_WARP || warp == F::O_WARP) {
        // ---------------- two threads that issue the products ----------------
        if (lane == 0) {
            const bool of_s = warp == F::S_WARP;
            constexpr uint32_t idesc_s = make_idesc_f16(false, 128, ROWS, false, false);
            constexpr uint32_t idesc_o = make_idesc_f16(false, 128, ROWS, true, true);
            const uint64_t desc_k = make_sdesc_sw128(sbase, 16, 1024);
            const uint64_t desc_v = make_sdesc_sw128(sbase + F::KTILE, kSwAtomBytes, 1024);
            const uint64_t desc_q = make_sdesc_sw128(sbase + F::Q_OFF, 16, 1024);
            const uint64_t desc_p = make_sdesc_sw128(sbase + F::P_OFF, kSwAtomBytes, 1024);
            int segments = 0;  // begun
            for (int g = 0, flags = 0; !(flags & kEnd); ++g) {
                const int buf = g & 1;
                if (!wait_bounded(bar((of_s ? F::B_KFULL : F::B_VFULL) + buf), (g >> 1) & 1, abort_flag))
                    break;
                flags = *reinterpret_cast<volatile int *>(&(of_s ? of_k : of_v)[g & 3].flags);
                const bool first = flags & kFirst;
                if (of_s) {
                    if (first && !wait_bounded(bar(F::B_QFULL), segments & 1, abort_flag))
                        break;
                    if (g >= 2 && !wait_bounded(bar(F::B_SFREE + buf), ((g >> 1) - 1) & 1, abort_flag))
                        break;
                    tc_fence_after();
                    const uint64_t kd = desc_k + static_cast<uint32_t>((buf * F::TILE) >> 4);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        umma_f16_ss(tmem + buf * ROWS,
                                    kd + static_cast<uint32_t>(((k >> 2) * kSwAtomBytes + (k & 3) * 32) >> 4),
                                    desc_q + static_cast<uint32_t>(((k >> 2) * F::BLK + (k & 3) * 32) >> 4), idesc_s,
                                    k > 0 ? 1u : 0u);
                    umma_commit(bar(F::B_SFULL + buf));
                } else {
                    if (!wait_bounded(bar(F::B_PFULL + buf), (g >> 1) & 1, abort_flag))
                        break;
                    if (first && segments > 0 && !wait_bounded(bar(F::B_OFREE), (segments - 1) & 1, abort_flag))
                        break;
                    tc_fence_after();
                    const uint64_t vd = desc_v + static_cast<uint32_t>((buf * F::TILE) >> 4);
                    const uint64_t pd = desc_p + static_cast<uint32_t>((g % F::PS * F::PTILE) >> 4);
#pragma unroll
                    for (int k = 0; k < F::STEP / 16; ++k)
                        umma_f16_ss(tmem + F::TM_O, vd + static_cast<uint32_t>((k * 2048) >> 4),
                                    pd + static_cast<uint32_t>((k * 2048) >> 4), idesc_o,
                                    first && k == 0 ? 0u : 1u);
                    umma_commit(bar(F::B_ODONE + buf));
                }
                segments += first;
            }
            // every product that this thread issued is done once this arrives
            umma_commit(bar(F::B_DRAIN + (of_s ? 0 : 1)));
            drain_bounded(bar(F::B_DRAIN + (of_s ? 0 : 1)), 0);
        }
    } else {
        // ---------------- softmax: four warps, of 128 keys or channels, for 16 rows ----------------
        constexpr int N = 16;
        const int quarter = warp & 3, t4 = t & 127, q0 = (warp >> 2) * N, barrier = 1 + (warp >> 2);
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + q0;
        float *row_scale = reinterpret_cast<float *>(smem + F::ROW_OFF) + q0, *row_m = row_scale + ROWS;
        int *row_last = reinterpret_cast<int *>(row_m + ROWS);  // the first key that the row does not see
        float *row_by = reinterpret_cast<float *>(row_last + ROWS);
        float *red = reinterpret_cast<float *>(smem + F::RED_OFF) + q0;
        const auto stop = [&](bool ok) { return named_bar_or(barrier, 128, !ok || *abort_flag != 0); };
        const auto arrive = [&](int x) {  // of the warp
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(x));
        };
        float l[N];
        int b = 0, head = 0, row0 = 0, least = 0;
        // unset: this thread's row has no reference; begun: O^T holds something
        bool unset = false, ok = true, begun = false;
        int g = 0;
        for (int flags = 0; !(flags & kEnd); ++g) {
            const int buf = g & 1;
            // A segment's first unit is known when its K is converted, whose product waits for Q; others
            // when theirs is there.  A warp whose wait failed meets the others, which do not know of it, at
            // the next two barriers; they leave at the second.
            const bool opens = flags & kLast || g == 0;
            if (!wait_warp(bar((opens ? F::B_KFULL : F::B_SFULL) + buf), (g >> 1) & 1, abort_flag)) {
                stop(false);
                stop(false);
                break;
            }
            const int4 info = *reinterpret_cast<const int4 *>(of_k + (g & 3));
            flags = info.x;
            if (opens) {
                if (stop(true)) {
                    stop(true);
                    break;
                }
                // ---- the segment's rows: to fp16, times a power of two ----
                b = info.z;
                head = info.w;
                row0 = of_k[g & 3].group * ROWS + q0;
                const int len = w.batch.length(b, log2_page);
                least = w.q.causal ? len - w.q.Nq + 1 : len;
                constexpr int PER = 128 / N, CH = D / PER;  // threads of a row, channels of a thread
                const int row = t4 / PER, c0 = t4 % PER * CH, abs_row = row0 + row;
                uint2 v[CH / 4];
#pragma unroll
                for (int i = 0; i < CH / 4; ++i)
                    v[i] = make_uint2(0, 0);
                int qi = 0;
                if (abs_row < w.R) {
                    const int hq = abs_row / w.q.Nq;
                    qi = abs_row % w.q.Nq;
                    const T *src = static_cast<const T *>(w.q.q) + b * w.q.batch_stride +
                                   static_cast<long long>(head * w.q.G + hq) * w.q.head_stride + qi * w.q.row_stride + c0;
#pragma unroll
                    for (int i = 0; i < CH / 4; ++i)
                        v[i] = *reinterpret_cast<const uint2 *>(src + 4 * i);
                }
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < CH / 4; ++i) {
                    const float2 y = DTypeTraits<T>::unpack(v[i].x), z = DTypeTraits<T>::unpack(v[i].y);
                    const float f[4] = {fabsf(y.x), fabsf(y.y), fabsf(z.x), fabsf(z.y)};
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (f[u] <= 3.402823466e38f)
                            top = fmaxf(top, f[u]);
                }
#pragma unroll
                for (int o = 1; o < PER; o <<= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const int e = top > 0.f ? max(static_cast<int>(__float_as_uint(top) >> 23) - 127 - 14, -100) : 0;
                const float by = cache::pow2f(-e);
#pragma unroll
                for (int i = 0; i < CH / 4; ++i) {
                    const float2 y = DTypeTraits<T>::unpack(v[i].x), z = DTypeTraits<T>::unpack(v[i].y);
                    cache::store_pair(sbase + F::Q_OFF + tile_offset<F::BLK>(q0 + row, c0 + 4 * i),
                                      DTypeTraits<__half>::pack(y.x * by, y.y * by),
                                      DTypeTraits<__half>::pack(z.x * by, z.y * by));
                }
                if (t4 % PER == 0) {
                    row_scale[row] = cache::pow2f(e) * w.scale_log2;
                    row_m[row] = 0.f;
                    row_last[row] = least + (w.q.causal ? qi : 0);
                }
                unset = t4 < N;
                begun = false;
#pragma unroll
                for (int q = 0; q < N; ++q)
                    l[q] = 0.f;
                fence_proxy_async_smem();
                named_bar_sync(barrier, 128);
                arrive(F::B_QFULL);
            }
            // ---- exponents; does any outgrow its reference? ----
            ok = !opens || wait_warp(bar(F::B_SFULL + buf), (g >> 1) & 1, abort_flag);
            tc_fence_after();
            uint32_t sc[N];
            tmem_ld16(lanes + buf * ROWS, sc);
            tc_fence_before();
            arrive(F::B_SFREE + buf);
            const unsigned copied = static_cast<unsigned>(flags) >> kBoxes;
            const int first = info.y << F::LOG2_STEP;
            const int key = copied >> (t4 >> w.log2_box) & 1 ? first + t4 : kNoKey;
            const bool masked = first + F::STEP > least || copied != all_boxes;
            float x[N];
#pragma unroll
            for (int q = 0; q < N; q += 4) {
                const float4 by = *reinterpret_cast<const float4 *>(row_scale + q);
                const float4 m = *reinterpret_cast<const float4 *>(row_m + q);
                const float2 a = ffma2(make_float2(__uint_as_float(sc[q]), __uint_as_float(sc[q + 1])),
                                       make_float2(by.x, by.y), make_float2(-m.x, -m.y));
                const float2 z = ffma2(make_float2(__uint_as_float(sc[q + 2]), __uint_as_float(sc[q + 3])),
                                       make_float2(by.z, by.w), make_float2(-m.z, -m.w));
                x[q] = a.x, x[q + 1] = a.y, x[q + 2] = z.x, x[q + 3] = z.y;
            }
            if (masked) {
#pragma unroll
                for (int q = 0; q < N; ++q)
                    x[q] = key < row_last[q] ? x[q] : -INFINITY;
            }
            float highest = unset ? INFINITY : -INFINITY;  // NaN moves no reference
#pragma unroll
            for (int q = 0; q < N; q += 2)
                highest = fmax3(highest, x[q], x[q + 1]);
            if (named_bar_or(barrier, 128, !ok || *abort_flag != 0 || highest > kMost)) {
                if (stop(ok))
                    break;
#pragma unroll
                for (int q = 0; q < N; ++q) {
                    float top = x[q];
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1)
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    if (lane == 0)
                        red[quarter * ROWS + q] = top;
                }
                named_bar_sync(barrier, 128);
                if (t4 < N) {
                    const float top = fmaxf(fmaxf(red[t4], red[ROWS + t4]), fmaxf(red[2 * ROWS + t4], red[3 * ROWS + t4]));
                    const float over = top - kAim;
                    const float up = unset ? (top == -INFINITY ? 0.f : over) : fmaxf(over, 0.f);
                    row_by[t4] = up;
                    red[t4] = unset ? 1.f : cache::ex2(-up);
                    row_m[t4] += up;
                    if (top > -INFINITY)
                        unset = false;
                }
                named_bar_sync(barrier, 128);
#pragma unroll
                for (int q = 0; q < N; ++q)
                    x[q] -= row_by[q];
                if (begun) {  // O^T and l by the references' steps
                    ok = wait_warp(bar(F::B_ODONE + (buf ^ 1)), ((g - 1) >> 1) & 1, abort_flag);
                    tc_fence_after();
                    tmem_ld16(lanes + F::TM_O, sc);
#pragma unroll
                    for (int q = 0; q < N; ++q) {
                        const float by = red[q];
                        sc[q] = __float_as_uint(__uint_as_float(sc[q]) * by);
                        l[q] *= by;
                    }
                    tmem_st16(lanes + F::TM_O, sc);
                    tmem_wait_st();
                }
            }
            // ---- P^T, as soon as an earlier product has read its tile ----
            uint32_t h[N / 2];
#pragma unroll
            for (int q = 0; q < N; q += 2) {
                const float2 p = make_float2(cache::ex2(x[q]), cache::ex2(x[q + 1]));
                const float2 sum = fadd2(make_float2(l[q], l[q + 1]), p);
                l[q] = sum.x;
                l[q + 1] = sum.y;
                h[q / 2] = DTypeTraits<__half>::pack(p.x, p.y);
            }
            if (g >= F::PS)
                ok = wait_warp(bar(F::B_ODONE + ((g - F::PS) & 1)), ((g - F::PS) >> 1) & 1, abort_flag) && ok;
            const uint32_t pt = sbase + F::P_OFF + g % F::PS * F::PTILE + t4 * 128, chunk = (q0 / 8) ^ (t4 & 7);
            st_shared_v4(pt + (chunk << 4), h[0], h[1], h[2], h[3]);
            st_shared_v4(pt + ((chunk ^ 1) << 4), h[4], h[5], h[6], h[7]);
            begun = true;
            fence_proxy_async_smem();
            tc_fence_before();
            if (ok)  // of the whole warp; without it the products' wait ends by itself
                arrive(F::B_PFULL + buf);

            if (flags & kLast) {
                // ---- the rows, or the block's part ----
                if (ok)
                    ok = wait_warp(bar(F::B_ODONE + buf), (g >> 1) & 1, abort_flag);
                if (stop(ok))
                    break;
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < N; ++q) {
                    float sum = l[q];
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1)
                        sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    if (lane == 0)
                        red[quarter * ROWS + q] = sum;
                }
                named_bar_sync(barrier, 128);
                const bool part = flags & (kHeadPart | kTailPart);
                const long long place = (2ll * blockIdx.x + (flags & kTailPart ? 1 : 0)) * ROWS + q0;
                const long long orow = (static_cast<long long>(b) * w.cache.heads + head) * w.R + row0;
                if (t4 < N) {
                    const float sum = red[t4] + red[ROWS + t4] + (red[2 * ROWS + t4] + red[3 * ROWS + t4]);
                    row_by[t4] = sum == 0.f ? 0.f : 1.f / sum;
                    const float m = row_m[t4];
                    if (row0 + t4 < w.R) {
                        if (part) {
                            w.part_m[place + t4] = unset ? -INFINITY : m;
                            w.part_l[place + t4] = sum;
                        } else if (lse != nullptr) {
                            lse[orow + t4] = sum == 0.f ? -INFINITY : (m + __log2f(sum)) * 0.6931471805599453f;
                        }
                    }
                }
                named_bar_sync(barrier, 128);
                tmem_ld16(lanes + F::TM_O, sc);
                tc_fence_before();
                arrive(F::B_OFREE);
#pragma unroll
                for (int q = 0; q < N; ++q)
                    if (t4 < D && row0 + q < w.R) {
                        const float y = __uint_as_float(sc[q]);
                        if (part)
                            w.part_o[(place + q) * D + t4] = y;
                        else
                            out[(orow + q) * D + t4] = to_type<T>(y * row_by[q]);
                    }
                named_bar_sync(barrier, 128);  // the rows' numbers are read
            }
        }
        tc_fence_before();
    }

    __syncthreads();
    if (warp == F::S_WARP) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, F::TM_COLS);
    }
}

}  // namespace cache4
}  // namespace fa
