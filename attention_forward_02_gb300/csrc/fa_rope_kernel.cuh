// fa_rope_kernel.cuh -- rotary positions of query and key rows on sm_103a, and their
// gradient: a pair of channels (a, b) at position p with angle t = p w becomes
// f (a cos t - b sin t, b cos t + a sin t); the gradient is the transpose, sin t with
// the other sign.
//
// What bounds it: each 16-bit value is read once and written once, six flops a pair beside
// it, so HBM does.  Sine and cosine depend on the row's position and the pair only: a
// thread takes four pairs of one row and goes through its heads with them.
//
// The angle is a fraction of a turn in 64-bit fixed point, position times turns[i] modulo
// 2^64: one whole product, exact for every position, where fp32 would lose a far position's
// angle and fp64 would be slow.  Its upper 32 bits, in half turns, go to sincospif.
#pragma once

#include "fa_cache_kernel.cuh"

namespace fa {
namespace rope {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // heads of a thread under way at once

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
};

// One thread: four pairs (or, behind the turned channels, eight channels that stay) of one
// row, and every `slots`-th head.  Pieces of four channels: of the pairs' first and second
// channels, or, interleaved, of pairs 0, 1 and 2, 3.
template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads)
    fa_rope_kernel(Rows q, Rows k, Turn turn, const int *positions, long long position_stride, int N,
                   int units, int slots, unsigned threads)
{
    cache::wait_ahead();
    cache::let_next();
    const unsigned i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= threads)
        return;
    const int unit = static_cast<int>(i % units);
    const unsigned x = i / units;
    const int slot = static_cast<int>(x % slots);
    const unsigned row = x / slots;
    const unsigned b = row / static_cast<unsigned>(N), n = row % static_cast<unsigned>(N);
    const int turning = turn.pairs / 4;
    const int p = positions ? positions[b * position_stride + n] : static_cast<int>(n);
    const bool turned = unit < turning && p >= 0;
    int at0, at1;  // the pieces' channels
    if (INTERLEAVED || unit >= turning) {
        at0 = 8 * unit;
        at1 = at0 + 4;
    } else {
        at0 = 4 * unit;
        at1 = turn.pairs + at0;
    }
    float cs[4], sn[4];
    if (turned) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const unsigned long long angle = turn.turns[4 * unit + j] * static_cast<unsigned long long>(p);
            const float half_turns = static_cast<float>(static_cast<int>(angle >> 32)) * 4.656612873077393e-10f;  // 2^-31
            sincospif(half_turns, &sn[j], &cs[j]);
            cs[j] *= turn.factor;
            sn[j] *= turn.backward ? -turn.factor : turn.factor;
        }
    }
    auto through = [&](const Rows &r, int first) {
        const T *src = static_cast<const T *>(r.x) + b * r.x_batch + n * r.x_row;
        T *dst = static_cast<T *>(r.y) + b * r.y_batch + n * r.y_row;
        for (int h0 = first; h0 < r.heads; h0 += kAhead * slots) {
            uint2 v[kAhead][2];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int h = h0 + u * slots;
                if (h < r.heads) {
                    v[u][0] = *reinterpret_cast<const uint2 *>(src + h * r.x_head + at0);
                    v[u][1] = *reinterpret_cast<const uint2 *>(src + h * r.x_head + at1);
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int h = h0 + u * slots;
                if (h >= r.heads)
                    break;
                if (turned) {
                    const uint32_t w[4] = {v[u][0].x, v[u][0].y, v[u][1].x, v[u][1].y};
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
                    v[u][0] = make_uint2(DTypeTraits<T>::pack(o[0], o[1]), DTypeTraits<T>::pack(o[2], o[3]));
                    v[u][1] = make_uint2(DTypeTraits<T>::pack(o[4], o[5]), DTypeTraits<T>::pack(o[6], o[7]));
                }
                *reinterpret_cast<uint2 *>(dst + h * r.y_head + at0) = v[u][0];
                *reinterpret_cast<uint2 *>(dst + h * r.y_head + at1) = v[u][1];
            }
        }
    };
    through(q, slot);
    // on with the keys where the queries' heads ended
    through(k, (slot + slots - q.heads % slots) % slots);
}

}  // namespace rope
}  // namespace fa
