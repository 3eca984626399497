// fa_cache4_decode_kernel.cuh -- decoding attention over the 4-bit paged cache on
// sm_103a: O = softmax(scale q K^T) V over the keys of a sequence.
#pragma once

#include "fa_cache4_kernel.cuh"

namespace fa {
namespace cache4 {

using cache::Queries;

// A block a query row: a thread a key for the scores of 128 keys, a thread a channel for
// the values.
constexpr int kSimpleThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kSimpleThreads)
    fa_cache4_decode_simple_kernel(Cache4 cache, Batch batch, Queries q, int d, float scale, T *__restrict__ out,
                                   float *__restrict__ lse)
{
    __shared__ float qs[128], p[kSimpleThreads], red[kSimpleThreads / 32];
    const int t = threadIdx.x;
    const int rows = cache.heads * q.G * q.Nq;
    const int b = blockIdx.x / rows, row = blockIdx.x % rows;
    const int hq = row / q.Nq, i = row % q.Nq, h = hq / q.G;
    const int len = batch.length(b, cache.log2_page);
    if (row == 0 && t == 0)
        batch.check_length(b, cache.log2_page);
    const int ctx = cache::context(q, len, i);
    if (t < d)
        qs[t] = static_cast<float>(
            static_cast<const T *>(q.q)[b * q.batch_stride + hq * q.head_stride + i * q.row_stride + t]);
    const int half = half_block(cache.page, d);
    float m = -INFINITY, l = 0.f, acc = 0.f;
    for (int k0 = 0; k0 < ctx; k0 += kSimpleThreads) {
        __syncthreads();
        const int key = k0 + t;
        float s = -INFINITY;
        if (key < ctx) {
            const int pg = batch.page(b, key >> cache.log2_page);
            if (pg < 0) {
                batch.bad();
            } else {
                const uint8_t *block = cache.data + (static_cast<size_t>(pg) * cache.heads + h) * (2 * half);
                const int r = key & (cache.page - 1);
                s = 0.f;
                for (int g = 0; g < d / kGroup; ++g) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(block + r * (d / 2) + 8 * g);
                    const uint32_t by = scale_pair(block[cache.page * (d / 2) + r * (d / kGroup) + g]);
                    uint32_t x[2][4];
                    halves8(w.x, x[0]);
                    halves8(w.y, x[1]);
                    for (int j = 0; j < 8; ++j) {
                        const float2 y = __half22float2(__hmul2(*reinterpret_cast<const __half2 *>(&x[j >> 2][j & 3]),
                                                                *reinterpret_cast<const __half2 *>(&by)));
                        s = fmaf(y.x, qs[kGroup * g + 2 * j], s);
                        s = fmaf(y.y, qs[kGroup * g + 2 * j + 1], s);
                    }
                }
                s *= scale;
            }
        }
        float top = s;
        for (int o = 16; o > 0; o >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if ((t & 31) == 0)
            red[t >> 5] = top;
        __syncthreads();
        for (int x = 0; x < kSimpleThreads / 32; ++x)
            top = fmaxf(top, red[x]);
        const float next = fmaxf(m, top), ref = next == -INFINITY ? 0.f : next;
        const float alpha = expf(m - ref);
        p[t] = expf(s - ref);
        __syncthreads();
        l *= alpha;
        acc *= alpha;
        m = next;
        const int n = min(kSimpleThreads, ctx - k0);
        for (int x = 0; x < n; ++x) {
            l += p[x];
            const int pg = batch.page(b, (k0 + x) >> cache.log2_page);
            if (t < d && pg >= 0) {
                const uint8_t *block = cache.data + (static_cast<size_t>(pg) * cache.heads + h) * (2 * half) + half;
                const int r = (k0 + x) & (cache.page - 1);
                uint32_t y[4];
                halves8(block[r * (d / 2) + t / 2], y);
                const float2 z = __half22float2(*reinterpret_cast<const __half2 *>(&y[0]));
                const uint32_t by = scale_pair(block[cache.page * (d / 2) + r * (d / kGroup) + t / kGroup]);
                acc = fmaf(p[x] * __half2float(__ushort_as_half(by & 0xFFFFu)), t & 1 ? z.y : z.x, acc);
            }
        }
    }
    const long long orow = static_cast<long long>(b) * rows + row;
    if (t < d)
        out[orow * d + t] = static_cast<T>(l > 0.f ? acc / l : 0.f);
    if (t == 0 && lse != nullptr)
        lse[orow] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace cache4
}  // namespace fa
