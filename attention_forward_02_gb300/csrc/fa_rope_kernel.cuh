// fa_rope_kernel.cuh -- rotary positions of query and key rows on sm_103a, and their
// gradient: a pair of channels (a, b) at position p with angle t = p w becomes
// f (a cos t - b sin t, b cos t + a sin t); the gradient is the transpose, sin t with
// the other sign.
//
// What bounds it: each 16-bit value is read once and written once, six flops a pair beside
// it, so HBM does.  Sine and cosine depend on the row's position and the pair only.  With
// many rows a thread computes those of four pairs of one row and goes through its heads
// with them: 58,800 rows of 40 heads of 128 take 180 us on the GPU, 1.2 GB, 98 % of the
// measured copy rate.  With few rows the heads have to be shared out among threads, and a
// block computes its rows' sines once for all of them.  40 heads of 128, bf16, sines a
// block / a thread, us on the GPU:
//     100 rows 2.7 / 3.4, 400 3.6 / 4.5, 1,000 5.6 / 5.9, 5,000 20.6 / 19.5, 12,000 44 / 41,
//     30,000 105 / 94; 2,500 rows of 5 heads of 96 5.4 / 4.0
// where the blocks' waits for positions and sines are no longer hidden by others.
//
// The angle is a fraction of a turn in 64-bit fixed point, position times turns[i] modulo
// 2^64: one whole product, exact for every position, where fp32 would lose a far position's
// angle and fp64 would be slow.  It goes to sincospif in half turns, rounded to fp32: 2^-24 of itself
// twice at most.  (Its upper 32 bits alone lost the angles of slow pairs near position 0: below
// 2^-32 of a turn they were 0.  What the lower ones cost does not show: rope_step 2.3 us on the GPU,
// rope_train 23.5, rope_prompts 181 with either.)
#pragma once

#include "fa_cache_kernel.cuh"

namespace fa {
namespace rope {

constexpr int kThreads = 256;
constexpr int kAhead = 4;             // heads of a thread under way at once
constexpr int kPairs = kThreads * 4;  // of a block's rows, at most: a unit has four

struct Rows {
    const void *x;
    void *y;
    long long x_batch, x_head, x_row, y_batch, y_head, y_row;
    int heads;
};
struct Turn {
    const unsigned long long *turns;
    int pairs;
    float factor;
    bool backward;

    // factor cos and factor sin of pair i at position p
    __device__ __forceinline__ void at(int i, int p, float &c, float &s) const
    {
        const unsigned long long angle = turns[i] * static_cast<unsigned long long>(static_cast<long long>(p));
        // both halves, each nearest zero: small angles keep their bits
        const int upper = static_cast<int>((angle + 0x80000000ull) >> 32), lower = static_cast<int>(angle);
        const float half_turns = fmaf(static_cast<float>(lower), 1.0842021724855044e-19f,  // 2^-63
                                      static_cast<float>(upper) * 4.656612873077393e-10f);  // 2^-31
        sincospif(half_turns, &s, &c);
        c *= factor;
        s *= backward ? -factor : factor;
    }
};
// All rows: a unit of one is four pairs, or, behind the turned channels, eight that stay.
struct Shape {
    const int *positions;
    long long position_stride;
    unsigned N, total;  // rows a batch, in all
    int units, slots;   // slots: threads of a block (a grid, with a thread a row) that share a row's unit

    __device__ __forceinline__ int position(unsigned b, unsigned n) const
    {
        return positions ? positions[b * position_stride + n] : static_cast<int>(n);
    }
};

// A unit's two pieces of four channels: the pairs' first and second ones, or, interleaved, pairs
// 0, 1 and 2, 3.
struct Piece {
    int at0, at1;
};
template <bool INTERLEAVED>
__device__ __forceinline__ Piece piece_of(int unit, int pairs)
{
    if (INTERLEAVED || unit >= pairs / 4)
        return {8 * unit, 8 * unit + 4};
    return {4 * unit, pairs + 4 * unit};
}

template <typename T, bool INTERLEAVED>
__device__ __forceinline__ void turn_unit(uint2 (&v)[2], const float (&cs)[4], const float (&sn)[4])
{
    const uint32_t w[4] = {v[0].x, v[0].y, v[1].x, v[1].y};
    float f[8], o[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 y = DTypeTraits<T>::unpack(w[j]);
        f[2 * j] = y.x;
        f[2 * j + 1] = y.y;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int a = INTERLEAVED ? 2 * j : j, c = INTERLEAVED ? 2 * j + 1 : j + 4;
        o[a] = f[a] * cs[j] - f[c] * sn[j];
        o[c] = f[c] * cs[j] + f[a] * sn[j];
    }
    v[0] = make_uint2(DTypeTraits<T>::pack(o[0], o[1]), DTypeTraits<T>::pack(o[2], o[3]));
    v[1] = make_uint2(DTypeTraits<T>::pack(o[4], o[5]), DTypeTraits<T>::pack(o[6], o[7]));
}

// Every step-th of a row's heads, the queries' and behind them the keys', kAhead at once: loads the
// next ones, and turns (or copies) and stores them.
template <typename T>
struct Heads {
    const T *from[2];
    T *to[2];
    long long from_step[2], to_step[2];
    int queries, all, step;
    Piece piece;
    uint2 v[kAhead][2];

    __device__ __forceinline__ Heads(const Rows &q, const Rows &k, unsigned b, unsigned n, int every, Piece p)
        : queries(q.heads), all(q.heads + k.heads), step(every), piece(p)
    {
        from[0] = static_cast<const T *>(q.x) + b * q.x_batch + n * q.x_row;
        from[1] = static_cast<const T *>(k.x) + b * k.x_batch + n * k.x_row - q.heads * k.x_head;
        to[0] = static_cast<T *>(q.y) + b * q.y_batch + n * q.y_row;
        to[1] = static_cast<T *>(k.y) + b * k.y_batch + n * k.y_row - q.heads * k.y_head;
        from_step[0] = q.x_head, from_step[1] = k.x_head, to_step[0] = q.y_head, to_step[1] = k.y_head;
    }
    __device__ __forceinline__ void load(int first)
    {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int h = first + u * step;
            if (h < all) {
                const T *x = h < queries ? from[0] + h * from_step[0] : from[1] + h * from_step[1];
                v[u][0] = *reinterpret_cast<const uint2 *>(x + piece.at0);
                v[u][1] = *reinterpret_cast<const uint2 *>(x + piece.at1);
            }
        }
    }
    template <bool INTERLEAVED>
    __device__ __forceinline__ void store(int first, bool turned, const float (&cs)[4], const float (&sn)[4])
    {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int h = first + u * step;
            if (h >= all)
                break;
            if (turned)
                turn_unit<T, INTERLEAVED>(v[u], cs, sn);
            T *y = h < queries ? to[0] + h * to_step[0] : to[1] + h * to_step[1];
            *reinterpret_cast<uint2 *>(y + piece.at0) = v[u][0];
            *reinterpret_cast<uint2 *>(y + piece.at1) = v[u][1];
        }
    }
};

// A thread a unit of a row, and of `slots` shares of its heads.
template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) fa_rope_kernel(Rows q, Rows k, Turn turn, Shape shape)
{
    cache::wait_ahead();
    cache::let_next();
    const unsigned i = blockIdx.x * kThreads + threadIdx.x;
    const int unit = static_cast<int>(i % shape.units);
    const unsigned x = i / shape.units;
    const int slot = static_cast<int>(x % shape.slots);
    const unsigned row = x / shape.slots;
    if (row >= shape.total)
        return;
    const unsigned b = row / shape.N, n = row % shape.N;
    const int p = shape.position(b, n);
    const bool turned = unit < turn.pairs / 4 && p >= 0;
    float cs[4], sn[4];
    if (turned) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            turn.at(4 * unit + j, p, cs[j], sn[j]);
    }
    Heads<T> heads(q, k, b, n, shape.slots, piece_of<INTERLEAVED>(unit, turn.pairs));
    for (int h = slot; h < heads.all; h += kAhead * shape.slots) {
        heads.load(h);
        heads.template store<INTERLEAVED>(h, turned, cs, sn);
    }
}

// A block a few rows, whose sines it computes once while its first heads are on their way; blocks
// in y share their heads.
template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) fa_rope_rows_kernel(Rows q, Rows k, Turn turn, Shape shape)
{
    __shared__ __align__(16) float cosines[kPairs], sines[kPairs];
    cache::wait_ahead();
    cache::let_next();
    const int places = kThreads / shape.units, rows = places / shape.slots;
    const int unit = threadIdx.x % shape.units, x = threadIdx.x / shape.units;
    const int own = x / shape.slots, step = shape.slots * gridDim.y;
    const int slot = x % shape.slots + blockIdx.y * shape.slots;
    const unsigned row0 = blockIdx.x * rows, row = row0 + own;
    const bool live = own < rows && row < shape.total;
    const unsigned b = live ? row / shape.N : 0, n = live ? row % shape.N : 0;
    Heads<T> heads(q, k, b, n, step, piece_of<INTERLEAVED>(unit, turn.pairs));
    if (live)
        heads.load(slot);
    for (int i = threadIdx.x; i < rows * turn.pairs; i += kThreads) {
        const unsigned r = row0 + i / turn.pairs;
        if (r >= shape.total)
            break;
        turn.at(i % turn.pairs, shape.position(r / shape.N, r % shape.N), cosines[i], sines[i]);
    }
    __syncthreads();
    if (!live)
        return;
    const bool turned = unit < turn.pairs / 4 && shape.position(b, n) >= 0;
    float cs[4], sn[4];
    if (turned) {
        const float4 c = *reinterpret_cast<const float4 *>(cosines + own * turn.pairs + 4 * unit);
        const float4 s = *reinterpret_cast<const float4 *>(sines + own * turn.pairs + 4 * unit);
        cs[0] = c.x, cs[1] = c.y, cs[2] = c.z, cs[3] = c.w;
        sn[0] = s.x, sn[1] = s.y, sn[2] = s.z, sn[3] = s.w;
    }
    for (int h = slot; h < heads.all;) {
        heads.template store<INTERLEAVED>(h, turned, cs, sn);
        h += kAhead * step;
        heads.load(h);
    }
}

}  // namespace rope
}  // namespace fa
