// fa_cache_kernel.cuh -- the 8-bit paged KV cache on sm_103a: writing new
// tokens into it, reading it back, and choosing pages by a cheap score.  The
// attention over it is in fa_cache_decode_kernel.cuh.
//
// A page holds `page` tokens of every KV head as 8-bit codes, with one scale
// for its K and one for its V per head.  Scales are powers of two: x / scale,
// code * scale and the ratio of two scales are then exact in fp32, and the only
// rounding of a value on its way in is the one to its 8-bit code.  An e4m3 code
// loses nothing by such a scale (its relative step does not depend on it); an
// int8 code loses at most the one bit by which amax may fall short of 127.
#pragma once

#include "fa_common.cuh"

namespace fa {
namespace cache {

constexpr int kLowestExp = -60;  // scales are at least 2^-60

// The cache's buffers as the kernels take them.
struct Cache {
    uint8_t *k, *v;
    float *k_scale, *v_scale;
    int8_t *k_mean;
    float *k_mean_scale;
    int num_pages, heads, page, log2_page;
};

// The batch: lengths and page numbers, in device memory.
struct Batch {
    const int *seq_lens;
    const int *table;
    long long table_stride;
    int max_pages, num_pages;
    unsigned int *status;

    __device__ void bad() const { atomicOr(status, kStatusBounds); }
    // Page number in slot `at` of sequence b; -1 if it is none.
    __device__ int page(int b, int at) const
    {
        if (at < 0 || at >= max_pages)
            return -1;
        const int p = table[b * table_stride + at];
        return p >= 0 && p < num_pages ? p : -1;
    }
    // Tokens of sequence b, within its page table.
    __device__ int length(int b, int log2_page) const
    {
        const long long cap = static_cast<long long>(max_pages) << log2_page;
        const int n = seq_lens[b];
        return n <= 0 ? 0 : static_cast<int>(n < cap ? n : cap);
    }
};

__device__ __forceinline__ float pow2f(int e)  // 2^e, -126 <= e <= 127
{
    return __int_as_float((e + 127) << 23);
}

// Smallest e >= kLowestExp with a 2^-e <= TOP, for a >= 0 finite.  With
// a = 1.f 2^E and TOP = 1.g 2^F, e is E - F, one more if f > g.
template <uint32_t TOP_FRACTION, int TOP_EXP>
__device__ __forceinline__ int scale_exp(float a)
{
    const uint32_t u = __float_as_uint(a);
    const int e = static_cast<int>(u >> 23) - 127 - TOP_EXP + ((u & 0x7FFFFFu) > TOP_FRACTION ? 1 : 0);
    return e < kLowestExp ? kLowestExp : e;  // zero and subnormal numbers have E = -127 here
}

__device__ __forceinline__ int int8_exp(float a) { return scale_exp<0x7E0000u, 6>(a); }  // 127 = 1.984375 2^6

__device__ __forceinline__ int round_int8(float x)
{
    return x == x ? __float2int_rn(fminf(fmaxf(x, -127.f), 127.f)) : 0;
}

struct E4M3 {
    static constexpr int kUnit = 512;  // codes are whole multiples of 1 / kUnit
    static __device__ __forceinline__ int exp_of(float a) { return scale_exp<0x600000u, 8>(a); }  // 448 = 1.75 2^8
    static __device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d)
    {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
        return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
    }
    // Two codes to fp16, exactly.
    static __device__ __forceinline__ uint32_t half2_of(uint16_t w)
    {
        uint32_t r;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(w));
        return r;
    }
    // Four codes to four fp16.
    static __device__ __forceinline__ void halves(uint32_t w, uint32_t &lo, uint32_t &hi)
    {
        lo = half2_of(static_cast<uint16_t>(w & 0xFFFFu));
        hi = half2_of(static_cast<uint16_t>(w >> 16));
    }
};

struct I8 {
    static constexpr int kUnit = 1;
    static __device__ __forceinline__ int exp_of(float a) { return int8_exp(a); }
    static __device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d)
    {
        return (round_int8(a) & 0xFF) | (round_int8(b) & 0xFF) << 8 | (round_int8(c) & 0xFF) << 16 |
               static_cast<uint32_t>(round_int8(d)) << 24;
    }
    // With its sign bit flipped a code is c + 128, which as the low byte of
    // 0x64.. is the fp16 1024 + c + 128; taking 1152 off leaves c, exactly.
    static __device__ __forceinline__ void halves(uint32_t w, uint32_t &lo, uint32_t &hi)
    {
        const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), off);
        const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), off);
        lo = *reinterpret_cast<const uint32_t *>(&x);
        hi = *reinterpret_cast<const uint32_t *>(&y);
    }
};

template <typename C>
__device__ __forceinline__ void decode4(uint32_t w, float (&f)[4])
{
    uint32_t lo, hi;
    C::halves(w, lo, hi);
    const float2 a = DTypeTraits<__half>::unpack(lo), b = DTypeTraits<__half>::unpack(hi);
    f[0] = a.x;
    f[1] = a.y;
    f[2] = b.x;
    f[3] = b.y;
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &x, float (&f)[8])
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = DTypeTraits<T>::unpack(w[i]);
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
}

// Largest finite magnitude of a and the values of f.
__device__ __forceinline__ float finite_max(float a, const float (&f)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = fabsf(f[i]);
        if (x <= 3.402823466e38f)  // neither infinite nor NaN
            a = fmaxf(a, x);
    }
    return a;
}

// ---------------------------------------------------------------------------
// Writing
//
// One block per (sequence, touched page, head, K or V): it owns the page's
// codes and scale, so nothing is shared and nothing is atomic in memory.  The
// new rows of a page (at most 128 x 128 16-bit values) are held in registers
// between the pass that finds amax and the one that encodes: one read, one
// write.  Thread t holds 8 columns (t % (d / 8)) of the rows t / (d / 8),
// + page / 8, ...; eight 16-byte loads in flight a thread.
constexpr int kWriteRows = 8;     // rows a thread
constexpr int kWriteThreads = 256;  // most threads: page = d = 128

struct NewRows {
    const void *x[2];  // K, V
    long long token_stride[2], head_stride[2];
    const int *cu;  // or NULL: `each` tokens a sequence
    int each, total;
};

__device__ __forceinline__ float block_max(float a, float *smem)
{
    const int warps = (blockDim.x + 31) >> 5;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
    __syncthreads();  // earlier reads of smem are done
    if ((threadIdx.x & 31) == 0)
        smem[threadIdx.x >> 5] = a;
    __syncthreads();
    a = smem[0];
    for (int w = 1; w < warps; ++w)
        a = fmaxf(a, smem[w]);
    return a;
}

template <typename T, typename C>
__global__ void __launch_bounds__(kWriteThreads) fa_cache_write_kernel(Cache cache, Batch batch, NewRows in, int d)
{
    __shared__ float red[kWriteThreads / 32];
    __shared__ int sums[128];
    const int b = blockIdx.z, h = blockIdx.y >> 1, which = blockIdx.y & 1;
    const int page = cache.page;
    const int groups = d / 8;              // threads a row
    const int stride = page / kWriteRows;  // rows between a thread's rows
    const bool live = threadIdx.x < static_cast<unsigned>(groups * stride);
    const int col = (threadIdx.x % groups) * 8, row0 = threadIdx.x / groups;
    int t0, n;
    if (in.cu != nullptr) {
        t0 = in.cu[b];
        n = in.cu[b + 1] - t0;
        if (t0 < 0 || t0 > in.total || n < 0 || n > in.total - t0) {
            if (threadIdx.x == 0)
                batch.bad();
            return;
        }
    } else {
        t0 = b * in.each;
        n = in.each;
    }
    if (n == 0)
        return;
    const long long had = max(batch.seq_lens[b], 0);  // tokens before
    const long long end = had + n;
    const long long last = (end - 1) >> cache.log2_page;
    const T *x = static_cast<const T *>(in.x[which]) + h * in.head_stride[which] + col;
    uint8_t *codes = which ? cache.v : cache.k;
    float *scales = which ? cache.v_scale : cache.k_scale;
    for (long long at = (had >> cache.log2_page) + blockIdx.x; at <= last; at += gridDim.x) {
        const int p = at < batch.max_pages ? batch.page(b, static_cast<int>(at)) : -1;
        if (p < 0) {
            if (threadIdx.x == 0)
                batch.bad();
            continue;
        }
        const long long base = at << cache.log2_page;  // position of the page's slot 0
        const int lo = static_cast<int>(max(had - base, 0ll));
        const int hi = static_cast<int>(min(end - base, static_cast<long long>(page)));
        uint4 raw[kWriteRows];
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < kWriteRows; ++i) {
            const int row = row0 + i * stride;
            raw[i] = make_uint4(0, 0, 0, 0);
            if (live && row >= lo && row < hi)
                raw[i] = __ldcs(reinterpret_cast<const uint4 *>(x + (t0 + (base - had) + row) * in.token_stride[which]));
        }
#pragma unroll
        for (int i = 0; i < kWriteRows; ++i) {
            float f[8];
            unpack8<T>(raw[i], f);
            a = finite_max(a, f);
        }
        const size_t ph = static_cast<size_t>(p) * cache.heads + h;
        const float old = lo > 0 ? scales[ph] : 0.f;
        a = block_max(a, red);  // every thread has read the old scale when it returns
        const float scale = fmaxf(old, pow2f(C::exp_of(a)));
        const float inv = 1.f / scale;
        uint8_t *dst = codes + ph * page * d + col;
        const bool mean = which == 0 && hi == page && cache.k_mean != nullptr;
        int sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < kWriteRows; ++i) {
            const int row = row0 + i * stride;
            uint2 c = make_uint2(0, 0);
            if (live && row >= lo && row < hi) {
                float f[8];
                unpack8<T>(raw[i], f);
                c.x = C::encode4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
                c.y = C::encode4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
                *reinterpret_cast<uint2 *>(dst + row * d) = c;
            } else if (live && row < lo && (scale > old || mean)) {
                c = *reinterpret_cast<const uint2 *>(dst + row * d);
                if (scale > old) {  // old codes at the new scale
                    const float r = old * inv;
                    float f[4], g[4];
                    decode4<C>(c.x, f);
                    decode4<C>(c.y, g);
                    c.x = C::encode4(f[0] * r, f[1] * r, f[2] * r, f[3] * r);
                    c.y = C::encode4(g[0] * r, g[1] * r, g[2] * r, g[3] * r);
                    *reinterpret_cast<uint2 *>(dst + row * d) = c;
                }
            }
            if (mean) {
                float f[4], g[4];
                decode4<C>(c.x, f);
                decode4<C>(c.y, g);
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // NaN converts to 0
                    sum[j] += __float2int_rn(f[j] * C::kUnit);
                    sum[4 + j] += __float2int_rn(g[j] * C::kUnit);
                }
            }
        }
        if (threadIdx.x == 0)
            scales[ph] = scale;
        if (mean) {
            // channel sums in units of 1 / kUnit: whole numbers below 2^25, so
            // their order does not matter
            for (int c = threadIdx.x; c < d; c += blockDim.x)
                sums[c] = 0;
            __syncthreads();
            if (live)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    atomicAdd(&sums[col + j], sum[j]);
            __syncthreads();
            const float unit = 1.f / (static_cast<float>(C::kUnit) * page);  // a power of two
            float m = 0.f;
            for (int c = threadIdx.x; c < d; c += blockDim.x)
                m = fmaxf(m, fabsf(static_cast<float>(sums[c]) * unit));
            m = block_max(m, red);
            const int e = int8_exp(m);
            const double by = static_cast<double>(unit) * pow2f(-e);
            for (int c = threadIdx.x; c < d; c += blockDim.x)
                cache.k_mean[ph * d + c] = static_cast<int8_t>(max(-127, min(127, __double2int_rn(sums[c] * by))));
            if (threadIdx.x == 0)
                cache.k_mean_scale[ph] = pow2f(e) * scale;
            __syncthreads();  // sums are free for the next page
        }
    }
}

// ---------------------------------------------------------------------------
// Reading back
//
// 16 codes (16 bytes) in, 16 values (32 bytes) out a thread and step; bound by
// the bytes it writes.
constexpr int kReadThreads = 256;
constexpr int kReadSteps = 4;

template <typename T, typename C>
__global__ void __launch_bounds__(kReadThreads)
    fa_cache_read_kernel(Cache cache, Batch batch, T *__restrict__ k, T *__restrict__ v, int N, int d, int chunks)
{
    // blockIdx.x = (b * heads + h) * chunks + chunk; y: K or V
    const int which = blockIdx.y;
    const long long bh = blockIdx.x / chunks;
    const int chunk = blockIdx.x % chunks;
    const int b = static_cast<int>(bh / cache.heads), h = static_cast<int>(bh % cache.heads);
    const int groups = d / 16;
    const long long vectors = static_cast<long long>(N) * groups;
    const int len = batch.length(b, cache.log2_page);
    const uint8_t *codes = which ? cache.v : cache.k;
    const float *scales = which ? cache.v_scale : cache.k_scale;
    T *out = (which ? v : k) + bh * N * d;
    const long long first = static_cast<long long>(chunk) * (kReadThreads * kReadSteps) + threadIdx.x;
    uint4 c[kReadSteps];
    float s[kReadSteps];
#pragma unroll
    for (int i = 0; i < kReadSteps; ++i) {
        const long long at = first + i * kReadThreads;
        c[i] = make_uint4(0, 0, 0, 0);
        s[i] = 0.f;
        const int t = static_cast<int>(at / groups);
        if (at < vectors && t < len) {
            const int p = batch.page(b, t >> cache.log2_page);
            if (p >= 0) {
                const size_t ph = static_cast<size_t>(p) * cache.heads + h;
                s[i] = scales[ph];
                c[i] = *reinterpret_cast<const uint4 *>(codes + (ph * cache.page + (t & (cache.page - 1))) * d +
                                                        (at % groups) * 16);
            } else {
                batch.bad();
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kReadSteps; ++i) {
        const long long at = first + i * kReadThreads;
        if (at >= vectors)
            break;
        const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
        uint32_t r[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float f[4];
            decode4<C>(w[j], f);
            r[2 * j] = s[i] > 0.f ? DTypeTraits<T>::pack(f[0] * s[i], f[1] * s[i]) : 0u;
            r[2 * j + 1] = s[i] > 0.f ? DTypeTraits<T>::pack(f[2] * s[i], f[3] * s[i]) : 0u;
        }
        uint4 *dst = reinterpret_cast<uint4 *>(out + at * 16);
        __stcs(dst, make_uint4(r[0], r[1], r[2], r[3]));
        __stcs(dst + 1, make_uint4(r[4], r[5], r[6], r[7]));
    }
}

// ---------------------------------------------------------------------------
// Choosing pages

// Query rows as the kernels take them.
struct Queries {
    const void *q;
    long long batch_stride, head_stride, row_stride;
    int G, Nq, causal;  // query heads a KV head, rows a head
};

// Keys that query i of a sequence of `len` keys sees.
__device__ __forceinline__ int context(const Queries &q, int len, int i)
{
    const int c = q.causal ? len - q.Nq + 1 + i : len;
    return c > 0 ? c : 0;
}

// Floats as unsigned numbers of the same order.
__device__ __forceinline__ uint32_t ordered(float f)
{
    if (f == 0.f)
        return 0x80000000u;  // -0 as +0
    const uint32_t u = __float_as_uint(f);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

// Scores of 64 pages of one (sequence, KV head) a block, for every query.  Four
// lanes share a page: each holds a quarter of its int8 mean and multiplies it
// with the same quarter of the int8 query rows (dp4a, int32), which lie in
// shared memory, `kScoreRows` at a time.
constexpr int kScoreThreads = 256;
constexpr int kScorePages = kScoreThreads / 4;
constexpr int kScoreRows = 64;

template <int D, typename T>
__global__ void __launch_bounds__(kScoreThreads)
    fa_cache_score_kernel(Cache cache, Batch batch, Queries q, uint32_t *__restrict__ scores, int slots)
{
    constexpr int QUARTER = D / 16;  // 32-bit words a lane
    __shared__ __align__(16) int q8[kScoreRows][D / 4];
    __shared__ float q8_scale[kScoreRows];
    const int b = blockIdx.z, h = blockIdx.y;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quarter = threadIdx.x & 3;
    const int len = batch.length(b, cache.log2_page);
    const int n = (context(q, len, q.Nq - 1) + cache.page - 1) >> cache.log2_page;  // of the longest context
    const int at = blockIdx.x * kScorePages + (threadIdx.x >> 2);
    if (static_cast<int>(blockIdx.x) * kScorePages >= n || n <= slots)
        return;  // no page here, or every page is chosen anyway
    int mean[QUARTER];
    float mean_scale = 0.f;
#pragma unroll
    for (int i = 0; i < QUARTER; ++i)
        mean[i] = 0;
    // a page that is not complete has no summary yet; it is the last of every
    // context that reaches it
    const bool whole = at < (len >> cache.log2_page);
    bool ok = false;
    if (whole) {
        const int p = batch.page(b, at);
        ok = p >= 0;
        if (ok) {
            const size_t ph = static_cast<size_t>(p) * cache.heads + h;
            mean_scale = cache.k_mean_scale[ph];
            const int2 *src = reinterpret_cast<const int2 *>(cache.k_mean + ph * D) + quarter * (QUARTER / 2);
#pragma unroll
            for (int i = 0; i < QUARTER / 2; ++i) {
                const int2 w = src[i];
                mean[2 * i] = w.x;
                mean[2 * i + 1] = w.y;
            }
        } else {
            batch.bad();
        }
    }
    for (int i = 0; i < q.Nq; ++i) {
        float best = -INFINITY;
        for (int g0 = 0; g0 < q.G; g0 += kScoreRows) {
            const int rows = min(kScoreRows, q.G - g0);
            __syncthreads();  // the rows before are read
            for (int g = warp; g < rows; g += kScoreThreads / 32) {
                const T *src = static_cast<const T *>(q.q) + b * q.batch_stride +
                               static_cast<long long>(h * q.G + g0 + g) * q.head_stride + i * q.row_stride;
                // lane l holds columns 4 l .. 4 l + 3
                float f[4] = {0.f, 0.f, 0.f, 0.f};
                if (lane < D / 4) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(src + 4 * lane);
                    const float2 x = DTypeTraits<T>::unpack(w.x), y = DTypeTraits<T>::unpack(w.y);
                    f[0] = x.x;
                    f[1] = x.y;
                    f[2] = y.x;
                    f[3] = y.y;
                }
                float a = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (fabsf(f[j]) <= 3.402823466e38f)
                        a = fmaxf(a, fabsf(f[j]));
#pragma unroll
                for (int off = 16; off > 0; off >>= 1)
                    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
                const int e = int8_exp(a);
                const float inv = pow2f(-e);
                if (lane < D / 4)
                    q8[g][lane] = static_cast<int>(I8::encode4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv));
                if (lane == 0)
                    q8_scale[g] = pow2f(e);
            }
            __syncthreads();
            for (int g = 0; g < rows; ++g) {
                int dot = 0;
#pragma unroll
                for (int w = 0; w < QUARTER; w += 2) {
                    const int2 x = *reinterpret_cast<const int2 *>(&q8[g][quarter * QUARTER + w]);
                    dot = __dp4a(mean[w], x.x, dot);
                    dot = __dp4a(mean[w + 1], x.y, dot);
                }
                dot += __shfl_xor_sync(0xffffffffu, dot, 1);
                dot += __shfl_xor_sync(0xffffffffu, dot, 2);
                // a whole number below 2^21, and powers of two: exact
                best = fmaxf(best, (static_cast<float>(dot) * q8_scale[g]) * mean_scale);
            }
        }
        if (quarter == 0 && at < n) {
            const long long seg = (static_cast<long long>(b) * cache.heads + h) * q.Nq + i;
            scores[seg * batch.max_pages + at] = ok ? ordered(best) : 0u;
        }
    }
}

// The `want` largest of the candidates' scores, ties to the lower page, with
// the kept pages, in ascending order.  One block a (sequence, KV head, query):
// the smallest chosen score by four 8-bit digits (a histogram of the scores
// that share the digits found so far), then one ordered pass that writes.
constexpr int kPickThreads = 256;

__global__ void __launch_bounds__(kPickThreads)
    fa_cache_pick_kernel(Cache cache, Batch batch, Queries q, const uint32_t *__restrict__ scores,
                         int *__restrict__ pages, int slots, int keep_first, int keep_last)
{
    __shared__ int hist[256];
    __shared__ int above[kPickThreads / 32], equal[kPickThreads / 32];
    __shared__ int found[2];
    const long long seg = blockIdx.x;
    const int i = static_cast<int>(seg % q.Nq);
    const int b = static_cast<int>(seg / q.Nq / cache.heads);
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    int *out = pages + seg * slots;
    const int n = (context(q, batch.length(b, cache.log2_page), i) + cache.page - 1) >> cache.log2_page;
    if (n <= slots) {
        for (int j = t; j < slots; j += kPickThreads)
            out[j] = j < n ? j : -1;
        return;
    }
    const uint32_t *key = scores + seg * batch.max_pages;
    const int lo = keep_first, hi = n - keep_last;  // candidates
    int want = slots - keep_first - keep_last;      // < hi - lo
    uint32_t prefix = 0;
    for (int shift = 24; want > 0 && shift >= 0; shift -= 8) {
        hist[t] = 0;
        __syncthreads();
        for (int j = lo + t; j < hi; j += kPickThreads) {
            const uint32_t x = key[j];
            if (shift == 24 || (x >> (shift + 8)) == prefix)
                atomicAdd(&hist[(x >> shift) & 255u], 1);
        }
        __syncthreads();
        if (warp == 0) {
            // lane l: digits 255 - 8 l downwards; the digit where the running count reaches `want`
            int c[8], sum = 0;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                c[u] = hist[255 - 8 * lane - u];
                sum += c[u];
            }
            int before = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, before, off);
                if (lane >= off)
                    before += y;
            }
            before -= sum;
            if (before < want && before + sum >= want) {
                int u = 0;
                while (before + c[u] < want)
                    before += c[u++];
                found[0] = 255 - 8 * lane - u;
                found[1] = want - before;
            }
        }
        __syncthreads();
        prefix = (prefix << 8) | static_cast<uint32_t>(found[0]);
        want = found[1];  // still to take among the scores that begin with `prefix`
    }
    // ordered pass over all pages: kept, above the smallest chosen score, or
    // one of the first `want` that equal it
    const bool any = slots > keep_first + keep_last;
    int written = 0, taken = 0;
    for (int j0 = 0; j0 < n; j0 += kPickThreads) {
        const int j = j0 + t;
        bool in = false, eq = false;
        if (j < n) {
            if (j < lo || j >= hi) {
                in = true;
            } else if (any) {
                const uint32_t x = key[j];
                in = x > prefix;
                eq = x == prefix;
            }
        }
        const unsigned eqs = __ballot_sync(0xffffffffu, eq);
        if (lane == 0)
            equal[warp] = __popc(eqs);
        __syncthreads();
        int rank = taken + __popc(eqs & ((1u << lane) - 1u)), total = 0;
        for (int w = 0; w < kPickThreads / 32; ++w) {
            if (w < warp)
                rank += equal[w];
            total += equal[w];
        }
        taken += total;
        in = in || (eq && rank < want);
        const unsigned ins = __ballot_sync(0xffffffffu, in);
        if (lane == 0)
            above[warp] = __popc(ins);
        __syncthreads();
        int pos = written + __popc(ins & ((1u << lane) - 1u));
        total = 0;
        for (int w = 0; w < kPickThreads / 32; ++w) {
            if (w < warp)
                pos += above[w];
            total += above[w];
        }
        written += total;
        if (in)
            out[pos] = j;
    }
}

}  // namespace cache
}  // namespace fa
