// fa_cache4_running.cuh -- what a warp of the decoding kernels over the 4-bit cache holds of
// its query rows and their running softmax, and the arithmetic on 16-key tiles whose bytes are
// in registers.  A tile's 16 rows stand for its keys in the order of tile_key; a thread
// (g = lane / 4, c = lane % 4) has
//  - of K: D / 4 channels from c * D / 4 on, of rows g and g + 8, eight to a word;
//  - of V: v_column's channels of rows 2 c, 2 c + 1, + 8, eight to a word (four in the last of
//    d = 32 and 96).
//
// What is held in fewer than 32 bits: Q and P, as operands in fp16, the type in which K and V are
// exact.  Q is exact but for channels below 2^-28 of the row's largest (it is scaled by a
// power of two).  P keeps eleven bits under a reference 2^kAim below the row's largest weight, its
// sum is taken before the rounding: for fp16 outputs the error of o is 2.3e-4 of its rms where o's own
// rounding is 2.1e-4; for bf16 ones (1.7e-3) it does not show.  P as the sum of two fp16 numbers would
// take the second product twice.
#pragma once

#include "fa_cache4_kernel.cuh"
#include "fa_cache_decode_kernel.cuh"

namespace fa {
namespace cache4 {

using cache::kAim;
using cache::kMost;
using cache::kNoKey;
using cache::kTile;
using cache::Work;

// The key of a tile's row: reads of K from a page as it lies are free of bank conflicts, those of
// V at most two-way.
__device__ __forceinline__ int tile_key(int row) { return row ^ (row >> 2 & 1); }

__device__ __forceinline__ uint32_t times(uint32_t a, uint32_t b)
{
    const __half2 x = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&x);
}

// Words of eight consecutive channels of a key's K that a thread has: D / 4 channels from
// c * D / 4 on; and the one or two bytes of their scales, which scale_pairs spreads.  `codes`
// and `scales` are where its first ones lie.
template <int D>
__device__ __forceinline__ uint32_t k_scale_offset(int c)
{
    return D == 128 ? 2 * c : D == 96 ? 3 * c >> 1 : D == 64 ? c : c >> 1;
}
template <int D>
__device__ __forceinline__ void load_k(uint32_t codes, uint32_t scales, uint32_t (&w)[D / 32], uint32_t (&s)[D > 64 ? 2 : 1])
{
    s[0] = load_u8(scales);
    if constexpr (D > 64)
        s[1] = load_u8(scales + 1);
    if constexpr (D == 96) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            cache::load_words<1>(w + i, codes + 4 * i);
    } else {
        cache::load_words<D / 32>(w, codes);
    }
}
template <int D>
__device__ __forceinline__ void scale_pairs(const uint32_t (&s)[D > 64 ? 2 : 1], int c, uint32_t (&by)[D / 32])
{
    const uint32_t lo = s[0] * 0x800080u, hi = D > 64 ? s[D > 64 ? 1 : 0] * 0x800080u : lo;
    by[0] = lo;
    if constexpr (D == 64) {
        by[1] = lo;
    } else if constexpr (D == 96) {
        by[1] = c & 1 ? hi : lo;
        by[2] = hi;
    } else if constexpr (D == 128) {
        by[1] = lo;
        by[2] = by[3] = hi;
    }
}

// A thread's channels of a key's V: v_column's, eight to a word (four in the last of d = 32 and
// 96), and the scale byte of each word; as above.
template <int D>
__device__ __forceinline__ uint32_t v_code_offset(int g)
{
    return D == 128 ? 8 * g : D == 32 ? 2 * g : 4 * g;
}
template <int D>
__device__ __forceinline__ uint32_t v_scale_offset(int g)
{
    return D == 128 ? g : D == 32 ? g >> 2 : g >> 1;
}
template <int D>
__device__ __forceinline__ void load_v(uint32_t codes, uint32_t scales, int g, uint32_t (&w)[(D + 63) / 64],
                                       uint32_t (&s)[(D + 63) / 64])
{
    s[0] = load_u8(scales);
    if constexpr (D == 128) {
        cache::load_words<2>(w, codes);
        s[1] = s[0];
    } else if constexpr (D == 96) {
        cache::load_words<1>(w, codes);
        w[1] = load_u16(codes + 32 - 2 * g);
        s[1] = load_u8(scales + 4 + (g >> 2) - (g >> 1));
    } else if constexpr (D == 64) {
        cache::load_words<1>(w, codes);
    } else {
        w[0] = load_u16(codes);
    }
}

// ROWS query rows: 4 (twice in the eight columns of a product), 8, or 16 (two products).
template <int D, int ROWS, typename T>
struct Running {
    static constexpr int NT = ROWS == 16 ? 2 : 1;          // tiles of eight columns
    static constexpr bool PAIRS = ROWS == 4;               // columns are four rows twice
    static constexpr int KW = D / 16;                      // steps of the first product
    static constexpr int TILES = PAIRS ? D / 32 : D / 16;  // of O^T
    static constexpr int VX = (D + 63) / 64;               // words of a key's V
    static constexpr int KS = D > 64 ? 2 : 1;              // scale bytes of a key's K

    const int g, c;
    const int key_row;      // key of row g
    const int v_row[2];     // keys of rows 2 c, 2 c + 1
    const uint32_t of_first, of_second;  // bytes of a key pair's P that a column of first (second) channels
                                         // takes of the first and second key
    // Q^T operand: of query rows g (+ 8), their d in the order of the thread's K words; in
    // registers for eight rows, for sixteen in shared memory of the lane's own, 16 bytes a step
    uint32_t qb[NT == 1 ? KW : 1][2];
    const uint32_t q_own;
    float qf[NT][2];      // per query row 2 c, 2 c + 1 (+ 8): scale to log2 units
    uint32_t behind = 0;  // ... keys that it sees beyond `least`, a byte each
    float m[NT][2], l[NT][2], acc[TILES][NT][4];
    int least = 0, most = 0;  // keys that all rows see (negative: the first ones see none), that any row sees
    bool fresh = true;        // some row may have no reference yet
    uint32_t unset = 0;       // ... a bit each of the thread's

    __device__ __forceinline__ Running(int lane, uint32_t q_at)
        : g(lane >> 2), c(lane & 3), key_row(tile_key(lane >> 2)), v_row{tile_key(2 * (lane & 3)), tile_key(2 * (lane & 3) + 1)},
          of_first(lane < 16 ? 0x4410u : 0x1044u), of_second(lane < 16 ? 0x4432u : 0x3244u), q_own(q_at)
    {
    }

    __device__ __forceinline__ int limit(int nt, int u) const
    {
        return least + static_cast<int>((behind >> (8 * (2 * nt + u))) & 255u);
    }

    // Begins with rows row0 .. of KV head `head` of a sequence of `len` keys.
    __device__ __forceinline__ void open(const Work &w, int b, int head, int row0, int len)
    {
        most = len;
        least = w.q.causal ? most - w.q.Nq + 1 : most;
        behind = 0;
        fresh = true;
        unset = (1u << (2 * NT)) - 1u;
        uint2 rows_q[NT][KW];
        int extra[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = row0 + nt * 8 + (PAIRS ? g & 3 : g);
            const int hq = row / w.q.Nq, qi = row % w.q.Nq;
            extra[nt] = w.q.causal ? qi : 0;
            const T *src = static_cast<const T *>(w.q.q) + b * w.q.batch_stride +
                           static_cast<long long>(head * w.q.G + hq) * w.q.head_stride + qi * w.q.row_stride + c * (D / 4);
#pragma unroll
            for (int s = 0; s < KW; ++s) {
                rows_q[nt][s] = make_uint2(0, 0);
                if (row < w.R)
                    rows_q[nt][s] = *reinterpret_cast<const uint2 *>(src + 4 * s);
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const uint2(&x)[KW] = rows_q[nt];
            float top = 0.f;
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
            const float by = cache::pow2f(-e);
#pragma unroll
            for (int s = 0; s < KW; ++s) {
                const float2 y = DTypeTraits<T>::unpack(x[s].x), z = DTypeTraits<T>::unpack(x[s].y);
                const uint32_t q0 = DTypeTraits<__half>::pack(y.x * by, y.y * by);
                const uint32_t q1 = DTypeTraits<__half>::pack(z.x * by, z.y * by);
                if constexpr (NT == 1) {
                    qb[s][0] = q0;
                    qb[s][1] = q1;
                } else {
                    cache::store_pair(q_own + s * 512 + nt * 8, q0, q1);
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                qf[nt][u] = cache::pow2f(__shfl_sync(0xffffffffu, e, 8 * c + 4 * u)) * w.scale_log2;
                behind |= __shfl_sync(0xffffffffu, extra[nt], 8 * c + 4 * u) << (8 * (2 * nt + u));
                m[nt][u] = 0.f;
                l[nt][u] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < TILES; ++j)
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    acc[j][nt][u] = 0.f;
        }
    }

    // S^T = K Q^T of J tiles: codes of each word, scale bytes.
    template <int J>
    __device__ __forceinline__ void scores(const uint32_t (&kw)[J][2][D / 32], const uint32_t (&ks)[J][2][KS],
                                           float (&e)[J][NT][4]) const
    {
        uint32_t by[J][2][D / 32];
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int r = 0; r < 2; ++r)
                scale_pairs<D>(ks[j][r], c, by[j][r]);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    e[j][nt][u] = 0.f;
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
            uint32_t h[J][2][4];
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    halves8(kw[j][r][x], h[j][r]);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        h[j][r][i] = times(h[j][r][i], by[j][r][x]);
                }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int s = 2 * x + y;
                uint32_t z[2 * NT];
                if constexpr (NT == 1) {
                    z[0] = qb[s][0];
                    z[1] = qb[s][1];
                } else {
                    cache::load_words<4>(z, q_own + s * 512);
                }
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        cache::mma_f16(e[j][nt], h[j][0][2 * y], h[j][1][2 * y], h[j][0][2 * y + 1], h[j][1][2 * y + 1],
                                       z[2 * nt], z[2 * nt + 1]);
            }
        }
    }

    // Their weights, as operand of the second product.  key0: position of each tile's first key.
    template <int J>
    __device__ __forceinline__ void weights(float (&e)[J][NT][4], const int (&key0)[J], bool masked, uint32_t (&pb)[J][NT][2])
    {
        // ---- exponents of P, masks; does any outgrow its reference? ----
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float2 by = make_float2(qf[nt][0], qf[nt][1]), from = make_float2(-m[nt][0], -m[nt][1]);
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int u = 0; u < 4; u += 2) {
                    const float2 x = ffma2(make_float2(e[j][nt][u], e[j][nt][u + 1]), by, from);
                    e[j][nt][u] = x.x;
                    e[j][nt][u + 1] = x.y;
                }
        }
        if (masked) {
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (key0[j] + key_row + 8 * (u >> 1) >= limit(nt, u & 1))
                            e[j][nt][u] = -INFINITY;
        }
        float highest = fresh ? INFINITY : -INFINITY;  // NaN moves no reference
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int u = 0; u < 4; u += 2)
                    highest = fmax3(highest, e[j][nt][u], e[j][nt][u + 1]);
        if (__any_sync(0xffffffffu, highest > kMost)) {
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
                    const float alpha = unset & bit ? 1.f : cache::ex2(-up);
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
                    for (int j = 0; j < TILES; ++j) {
                        acc[j][nt][u] *= alpha;
                        acc[j][nt][u + 2] *= alpha;
                    }
                }
            fresh = __any_sync(0xffffffffu, unset != 0);
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float(&p)[4] = e[j][nt];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    p[u] = cache::ex2(p[u]);
                const float2 sum = fadd2(make_float2(l[nt][0], l[nt][1]),
                                         fadd2(make_float2(p[0], p[1]), make_float2(p[2], p[3])));
                l[nt][0] = sum.x;
                l[nt][1] = sum.y;
                pb[j][nt][0] = cache::transpose8(DTypeTraits<__half>::pack(p[0], p[1]));
                pb[j][nt][1] = cache::transpose8(DTypeTraits<__half>::pack(p[2], p[3]));
            }
        }
    }

    // O^T += V^T P^T of a tile: codes and scale bytes of each word.
    __device__ __forceinline__ void values(const uint32_t (&vw)[4][VX], uint32_t (&vs)[4][VX], const uint32_t (&pb)[NT][2],
                                           int key0, bool masked)
    {
        if (masked) {
            // bytes behind the last key are whatever the page held: codes are finite, a scale
            // need not be
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (key0 + v_row[r & 1] + 8 * (r >> 1) >= most)
#pragma unroll
                    for (int x = 0; x < VX; ++x)
                        vs[r][x] = 0;
        }
        if constexpr (PAIRS) {
            // a pair's two channels as two terms of the product, each with the key's weight for its
            // own columns and 0 for the other's
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t b0 = __byte_perm(pb[0][r], 0, of_first), b1 = __byte_perm(pb[0][r], 0, of_second);
#pragma unroll
                for (int x = 0; x < VX; ++x) {
                    const bool half_word = x == VX - 1 && D % 64 != 0;
                    uint32_t h[2][4];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        halves8(vw[2 * r + y][x], h[y]);
#pragma unroll
                        for (int i = 0; i < (half_word ? 2 : 4); ++i)
                            h[y][i] = times(h[y][i], vs[2 * r + y][x] * 0x800080u);
                    }
#pragma unroll
                    for (int i = 0; i < (half_word ? 1 : 2); ++i)
                        cache::mma_f16(acc[2 * x + i][0], h[0][2 * i], h[0][2 * i + 1], h[1][2 * i], h[1][2 * i + 1], b0,
                                       b1);
                }
            }
        } else {
#pragma unroll
            for (int x = 0; x < VX; ++x) {
                // the channels of a word, of keys 2 c and 2 c + 1, and of the two 8 behind them
                const bool half_word = x == VX - 1 && D % 64 != 0;
                uint32_t even[2][4], odd[2][4];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t a = vw[2 * r][x], z = vw[2 * r + 1][x];
                    const uint32_t by = vs[2 * r][x] * 0x80u + vs[2 * r + 1][x] * 0x800000u;
                    halves8((a & 0x0F0F0F0Fu) | (z << 4 & 0xF0F0F0F0u), even[r]);
                    halves8((a >> 4 & 0x0F0F0F0Fu) | (z & 0xF0F0F0F0u), odd[r]);
#pragma unroll
                    for (int i = 0; i < (half_word ? 2 : 4); ++i) {
                        even[r][i] = times(even[r][i], by);
                        odd[r][i] = times(odd[r][i], by);
                    }
                }
#pragma unroll
                for (int i = 0; i < (half_word ? 2 : 4); ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        cache::mma_f16(acc[4 * x + i][nt], even[0][i], odd[0][i], even[1][i], odd[1][i], pb[nt][0],
                                       pb[nt][1]);
            }
        }
    }
};

}  // namespace cache4
}  // namespace fa
