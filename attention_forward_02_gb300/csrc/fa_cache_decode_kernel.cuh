// fa_cache_decode_kernel.cuh -- decoding attention over the 8-bit paged cache
// on sm_103a: O = softmax(scale q K^T) V with K = k_scale * codes, V likewise,
// over all keys of a sequence or over listed pages only.
#pragma once

#include "fa_cache_kernel.cuh"

namespace fa {
namespace cache {

// One warp a query row: 32 keys at a time, lane l the score of key l, then all
// lanes the columns l, l + 32, ... of P V.
template <int D, typename T, typename C>
__global__ void __launch_bounds__(128)
    fa_cache_decode_kernel(Cache cache, Batch batch, Queries q, const int *__restrict__ pages, int slots,
                           T *__restrict__ out, float *__restrict__ lse, long long rows, int Hq, float scale_log2)
{
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows)
        return;
    const int i = static_cast<int>(row % q.Nq), hq = static_cast<int>(row / q.Nq % Hq);
    const int b = static_cast<int>(row / q.Nq / Hq), h = hq / q.G;
    const int ctx = context(q, batch.length(b, cache.log2_page), i);
    const int n = (ctx + cache.page - 1) >> cache.log2_page;
    const int count = pages ? min(n, slots) : n;
    const int *list = pages ? pages + ((static_cast<long long>(b) * cache.heads + h) * q.Nq + i) * slots : nullptr;
    const T *src = static_cast<const T *>(q.q) + b * q.batch_stride + hq * q.head_stride + i * q.row_stride;
    float m = -INFINITY, l = 0.f, o[D / 32];
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
        o[c] = 0.f;
    for (int s = 0; s < count; ++s) {
        const int at = list ? list[s] : s;
        if (at < 0)
            continue;
        const int p = at < n ? batch.page(b, at) : -1;
        if (p < 0) {
            batch.bad();
            continue;
        }
        const size_t ph = static_cast<size_t>(p) * cache.heads + h;
        const uint8_t *k = cache.k + ph * cache.page * D, *v = cache.v + ph * cache.page * D;
        const float ks = cache.k_scale[ph] * scale_log2, vs = cache.v_scale[ph];
        const int keys = min(cache.page, ctx - (at << cache.log2_page));
        for (int j0 = 0; j0 < keys; j0 += 32) {
            float x = -INFINITY;
            if (j0 + lane < keys) {
                float dot = 0.f;
                for (int c = 0; c < D; c += 4) {
                    float f[4];
                    decode4<C>(*reinterpret_cast<const uint32_t *>(k + (j0 + lane) * D + c), f);
                    const uint2 w = *reinterpret_cast<const uint2 *>(src + c);
                    const float2 a = DTypeTraits<T>::unpack(w.x), e = DTypeTraits<T>::unpack(w.y);
                    dot = fmaf(a.x, f[0], fmaf(a.y, f[1], fmaf(e.x, f[2], fmaf(e.y, f[3], dot))));
                }
                x = dot * ks;
            }
            float top = x;
            for (int off = 16; off > 0; off >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float m_new = fmaxf(m, top);
            const float ref = m_new == -INFINITY ? 0.f : m_new;
            const float alpha = exp2f(m - ref), e = exp2f(x - ref);
            m = m_new;
            l = l * alpha + e;
            for (int c = 0; c < D / 32; ++c)
                o[c] *= alpha;
            for (int j = 0; j < 32 && j0 + j < keys; ++j) {
                const float w = __shfl_sync(0xffffffffu, e, j) * vs;
                for (int c = 0; c < D / 32; ++c) {
                    float f[4];
                    decode4<C>(v[(j0 + j) * D + c * 32 + lane], f);
                    o[c] = fmaf(w, f[0], o[c]);
                }
            }
        }
    }
    for (int off = 16; off > 0; off >>= 1)
        l += __shfl_xor_sync(0xffffffffu, l, off);
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    for (int c = 0; c < D / 32; ++c) {
        const uint32_t r = DTypeTraits<T>::pack(o[c] * inv, 0.f);
        reinterpret_cast<uint16_t *>(out)[row * D + c * 32 + lane] = static_cast<uint16_t>(r);
    }
    if (lse != nullptr && lane == 0)
        lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace cache
}  // namespace fa
