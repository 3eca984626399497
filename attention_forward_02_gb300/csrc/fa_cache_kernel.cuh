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
    // Reports a length that length() cuts; one thread of a call does it for a sequence.
    __device__ void check_length(int b, int log2_page) const
    {
        const int n = seq_lens[b];
        if (n < 0 || n > static_cast<long long>(max_pages) << log2_page)
            bad();
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

// Dependent launches.  A kernel launched so may begin before the one ahead of it
// in the stream has ended: it calls wait_ahead() before it touches memory, which
// returns when that one has completed and its writes are visible.  let_next() lets
// the next such launch begin; it is called after wait_ahead(), so whatever a later
// kernel reads before its own wait was complete before this one's work began.
__device__ __forceinline__ void wait_ahead() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// x 2^-s rounded to the nearest whole number (ties to even), for |x| < 2^25 and a
// result of at most 127.
__device__ __forceinline__ int scale_round(int x, int s)
{
    if (s <= 0)
        return x * (1 << min(-s, 30));  // exact; x = 0 where s is far below
    if (s > 26)
        return 0;
    const int q = x >> s, rest = x - q * (1 << s), half = 1 << (s - 1);
    return q + (rest > half || (rest == half && (q & 1)) ? 1 : 0);
}

struct E4M3 {
    static constexpr int kUnit = 512, kLog2Unit = 9;  // codes are whole multiples of 1 / kUnit
    static __device__ __forceinline__ int exp_of(float a) { return scale_exp<0x600000u, 8>(a); }  // 448 = 1.75 2^8
    static __device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d)
    {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
        return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
    }
    // Finite values, scaled on the way.
    static __device__ __forceinline__ uint32_t encode4_finite(float a, float b, float c, float d, float inv)
    {
        return encode4(a * inv, b * inv, c * inv, d * inv);
    }
    // The same on two pairs of fp16: the scaled value has fp16's 11 bits, or is
    // below the smallest code (2^-9) by far, so it is exact where it matters.
    static __device__ __forceinline__ uint32_t encode4_half(uint32_t ab, uint32_t cd, __half2 inv)
    {
        const __half2 x = __hmul2(*reinterpret_cast<const __half2 *>(&ab), inv);
        const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&cd), inv);
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(lo) : "r"(*reinterpret_cast<const uint32_t *>(&x)));
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hi) : "r"(*reinterpret_cast<const uint32_t *>(&y)));
        return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
    }
    // Four codes to four fp16, exactly.
    static __device__ __forceinline__ void halves(uint32_t w, uint32_t &lo, uint32_t &hi)
    {
        asm("{\n\t.reg .b16 l, h;\n\t"
            "mov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=&r"(lo), "=r"(hi)
            : "r"(w));
    }
};

struct I8 {
    static constexpr int kUnit = 1, kLog2Unit = 0;
    static __device__ __forceinline__ int exp_of(float a) { return int8_exp(a); }
    static __device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d)
    {
        return (round_int8(a) & 0xFF) | (round_int8(b) & 0xFF) << 8 | (round_int8(c) & 0xFF) << 16 |
               static_cast<uint32_t>(round_int8(d)) << 24;
    }
    // Finite values of at most 127 once scaled: 1.5 2^23 + x has x rounded to the
    // nearest whole number (ties to even) in its low bits, two's complement.
    static __device__ __forceinline__ uint32_t encode4_finite(float a, float b, float c, float d, float inv)
    {
        const float k = 12582912.f;
        const uint32_t x = __byte_perm(__float_as_uint(fmaf(a, inv, k)), __float_as_uint(fmaf(b, inv, k)), 0x0040);
        const uint32_t y = __byte_perm(__float_as_uint(fmaf(c, inv, k)), __float_as_uint(fmaf(d, inv, k)), 0x0040);
        return __byte_perm(x, y, 0x5410);
    }
    // The same on two pairs of fp16, with 1.5 2^10: one rounding, in the fused addition.
    static __device__ __forceinline__ uint32_t encode4_half(uint32_t ab, uint32_t cd, __half2 inv)
    {
        const __half2 k = __halves2half2(__ushort_as_half(0x6600), __ushort_as_half(0x6600));
        const __half2 x = __hfma2(*reinterpret_cast<const __half2 *>(&ab), inv, k);
        const __half2 y = __hfma2(*reinterpret_cast<const __half2 *>(&cd), inv, k);
        return __byte_perm(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y), 0x6420);
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
// More new rows than sequences, as in prompts: one block per (touched page, head, K
// or V).  It owns the page's codes and scale, so nothing is shared and nothing is
// atomic in memory.  The
// new rows of a page (at most 128 x 128 16-bit values) are held in registers
// between the pass that finds amax and the one that encodes: one read, one
// write.  Thread t holds 8 columns (t % (d / 8)) of the rows t / (d / 8),
// + page / 8, ...; eight 16-byte loads in flight a thread.  For long prompts the
// instructions bound it, so amax is taken on pairs of 16-bit values and fp16 is
// encoded in pairs; pages with infinities or NaN, which the maximum shows, and
// scales beyond fp16's range go another way.  58,800 tokens of 8 heads of 128 (361 MB):
// from fp16 to int8 62 us on the GPU, 5.8 TB/s, 86 % of the measured copy rate, to e4m3
// 64; from bf16, which is encoded one by one in fp32, 66 and 67.
constexpr int kWriteRows = 8;       // rows a thread
constexpr int kWriteThreads = 256;  // most threads: page = d = 128

struct NewRows {
    const void *x[2];  // K, V
    long long token_stride[2], head_stride[2];
    const int *cu;  // or NULL: `each` tokens a sequence
    int each, total, batch;

    // First row and rows of sequence b; false if its offsets are none.
    __device__ bool tokens(int b, int &first, int &count) const
    {
        first = cu ? cu[b] : b * each;
        count = cu ? cu[b + 1] - first : each;
        return first >= 0 && first <= total && count >= 0 && count <= total - first;
    }
};

// Larger magnitudes of two pairs (NaN if one is; the sign means nothing).
template <typename T>
__device__ __forceinline__ uint32_t max_magnitude2(uint32_t a, uint32_t b)
{
    uint32_t d;
    if (DTypeTraits<T>::kBF16)
        asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The block's largest x (of unsigned numbers).
__device__ __forceinline__ uint32_t block_max(uint32_t x, uint32_t *smem)
{
    const int warps = (blockDim.x + 31) >> 5;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        x = max(x, __shfl_xor_sync(0xffffffffu, x, off));
    __syncthreads();  // earlier reads of smem are done
    if ((threadIdx.x & 31) == 0)
        smem[threadIdx.x >> 5] = x;
    __syncthreads();
    x = smem[0];
    for (int w = 1; w < warps; ++w)
        x = max(x, smem[w]);
    return x;
}

// Sums of a thread's codes down its rows, for its eight columns, in units of
// 1 / kUnit; exact (int8: two biased 16-bit sums a word; e4m3: 21 bits in fp32).
template <typename C>
struct ColumnSums;
template <>
struct ColumnSums<I8> {
    uint32_t even[2] = {0, 0}, odd[2] = {0, 0};
    int rows = 0;
    __device__ __forceinline__ void add(const uint2 &c, bool)
    {
        const uint32_t w[2] = {c.x ^ 0x80808080u, c.y ^ 0x80808080u};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            even[i] += w[i] & 0x00FF00FFu;
            odd[i] += (w[i] >> 8) & 0x00FF00FFu;
        }
        ++rows;
    }
    __device__ __forceinline__ int sum(int j) const
    {
        const uint32_t x = j & 1 ? odd[j >> 2] : even[j >> 2];
        return static_cast<int>(j & 2 ? x >> 16 : x & 0xFFFFu) - 128 * rows;
    }
};
template <>
struct ColumnSums<E4M3> {
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    __device__ __forceinline__ void add(uint2 c, bool finite)
    {
        if (!finite) {  // NaN codes (all but the sign set) count as 0
            const uint32_t x = ((c.x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
            const uint32_t y = ((c.y & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
            c.x &= ~((x >> 7) * 0xFFu);
            c.y &= ~((y >> 7) * 0xFFu);
        }
        float f[4], g[4];
        decode4<E4M3>(c.x, f);
        decode4<E4M3>(c.y, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[j] += f[j];
            s[4 + j] += g[j];
        }
    }
    __device__ __forceinline__ int sum(int j) const { return __float2int_rn(s[j] * E4M3::kUnit); }
};

// The sequence of the `skip`-th touched page of the batch, and in `skip` which of the
// sequence's; -1 if there are fewer.  A warp counts the pages of 32 sequences at a
// time, with the offsets and lengths of 32 * AHEAD on their way: these loads are what
// a block with few rows waits for.  AHEAD of four takes 256 sequences with one prompt
// of 512 tokens among them from 29.7 to 24.5 us, 1,000 of 7 tokens from 49.3 to 33.0;
// up to 32 sequences, where it could only cost (prompts 62.5 -> 63.6), it is one.
template <int AHEAD>
__device__ __forceinline__ int touched_page(const Cache &cache, const Batch &batch, const NewRows &in, long long &skip)
{
    const int lane = threadIdx.x & 31;
    for (int b0 = 0; b0 < in.batch; b0 += 32 * AHEAD) {
        int count[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int x = b0 + 32 * u + lane;
            count[u] = 0;
            if (x < in.batch) {
                const long long had = batch.seq_lens[x];
                int t0, n;
                if (!in.tokens(x, t0, n) || (n > 0 && had < 0))
                    batch.bad();
                else if (n > 0)
                    count[u] = static_cast<int>(((had + n - 1) >> cache.log2_page) - (had >> cache.log2_page)) + 1;
            }
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            if (AHEAD > 1) {  // most of many chunks are only passed over
                const int all = __reduce_add_sync(0xffffffffu, count[u]);
                if (skip >= all) {
                    skip -= all;
                    continue;
                }
            }
            int incl = count[u];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off)
                    incl += y;
            }
            const unsigned here = __ballot_sync(0xffffffffu, skip < incl);
            if (here) {
                const int from = __ffs(here) - 1;
                skip -= __shfl_sync(0xffffffffu, incl - count[u], from);
                return b0 + 32 * u + from;
            }
            skip -= __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    return -1;
}

template <typename T, typename C>
__global__ void __launch_bounds__(kWriteThreads, 4) fa_cache_write_kernel(Cache cache, Batch batch, NewRows in, int d)
{
    __shared__ uint32_t red[kWriteThreads / 32];
    __shared__ int sums[128];
    const uint32_t infinity = DTypeTraits<T>::kBF16 ? 0x7F80u : 0x7C00u;
    const int h = blockIdx.y >> 1, which = blockIdx.y & 1;
    const int page = cache.page;
    const int groups = d / 8;              // threads a row
    const int stride = page / kWriteRows;  // rows between a thread's rows
    const bool live = threadIdx.x < static_cast<unsigned>(groups * stride);
    const int col = (threadIdx.x % groups) * 8, row0 = threadIdx.x / groups;
    long long skip = blockIdx.x;
    const int b = in.batch <= 32 ? touched_page<1>(cache, batch, in, skip) : touched_page<4>(cache, batch, in, skip);
    if (b < 0)
        return;  // fewer pages than blocks
    int t0, n;
    in.tokens(b, t0, n);
    const long long had = batch.seq_lens[b];  // tokens before
    const long long end = had + n;
    const long long token_stride = which ? in.token_stride[1] : in.token_stride[0];
    const T *x = static_cast<const T *>(which ? in.x[1] : in.x[0]) +
                 h * (which ? in.head_stride[1] : in.head_stride[0]) + col;
    uint8_t *codes = which ? cache.v : cache.k;
    float *scales = which ? cache.v_scale : cache.k_scale;
    const long long at = (had >> cache.log2_page) + skip;
    const int p = at < batch.max_pages ? batch.page(b, static_cast<int>(at)) : -1;
    if (p < 0) {
        if (threadIdx.x == 0)
            batch.bad();
        return;
    }
    const long long base = at << cache.log2_page;  // position of the page's slot 0
    const int lo = static_cast<int>(max(had - base, 0ll));
    const int hi = live ? static_cast<int>(min(end - base, static_cast<long long>(page))) : 0;
    const T *src = x + (t0 + (base - had) + row0) * token_stride;  // of slot row0, if that is new
    const long long step = stride * token_stride;
    const bool whole = lo == 0 && end - base >= page;  // every slot is new: no row of it needs a look
    uint4 raw[kWriteRows];
    uint32_t m = 0;
    if (whole && live) {
        const T *from = src;
#pragma unroll
        for (int i = 0; i < kWriteRows; ++i, from += step)
            raw[i] = __ldcs(reinterpret_cast<const uint4 *>(from));
    } else {
#pragma unroll
        for (int i = 0; i < kWriteRows; ++i) {
            const int row = row0 + i * stride;
            raw[i] = make_uint4(0, 0, 0, 0);
            if (row >= lo && row < hi)
                raw[i] = __ldcs(reinterpret_cast<const uint4 *>(src + i * step));
        }
    }
#pragma unroll
    for (int i = 0; i < kWriteRows; ++i) {
        m = max_magnitude2<T>(m, max_magnitude2<T>(raw[i].x, raw[i].y));
        m = max_magnitude2<T>(m, max_magnitude2<T>(raw[i].z, raw[i].w));
    }
    m &= 0x7FFF7FFFu;
    const size_t ph = static_cast<size_t>(p) * cache.heads + h;
    const float old = lo > 0 ? scales[ph] : 0.f;
    m = block_max(max(m & 0xFFFFu, m >> 16), red);  // every thread has read the old scale when it returns
    const bool finite = m < infinity;
    float a = DTypeTraits<T>::unpack(m).x;
    if (!finite) {
        a = 0.f;
#pragma unroll
        for (int i = 0; i < kWriteRows; ++i) {
            float f[8];
            unpack8<T>(raw[i], f);
            a = finite_max(a, f);
        }
        a = __uint_as_float(block_max(__float_as_uint(a), red));
    }
    const float scale = fmaxf(old, pow2f(C::exp_of(a)));
    const float inv = 1.f / scale;
    const bool pairs = finite && inv >= 6.103515625e-5f && inv <= 32768.f;  // a normal fp16 number
    const __half2 inv2 = __float2half2_rn(inv);
    uint8_t *dst = codes + ph * page * d + row0 * d + col;
    const bool mean = which == 0 && end - base >= page && cache.k_mean != nullptr;
    ColumnSums<C> sum;
    if (whole && finite && (DTypeTraits<T>::kBF16 || pairs)) {
        if (live) {
            uint8_t *to = dst;
#pragma unroll
            for (int i = 0; i < kWriteRows; ++i, to += stride * d) {
                uint2 c;
                if (DTypeTraits<T>::kBF16) {
                    float f[8];
                    unpack8<T>(raw[i], f);
                    c.x = C::encode4_finite(f[0], f[1], f[2], f[3], inv);
                    c.y = C::encode4_finite(f[4], f[5], f[6], f[7], inv);
                } else {
                    c.x = C::encode4_half(raw[i].x, raw[i].y, inv2);
                    c.y = C::encode4_half(raw[i].z, raw[i].w, inv2);
                }
                *reinterpret_cast<uint2 *>(to) = c;
                if (mean)
                    sum.add(c, true);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kWriteRows; ++i) {
            const int row = row0 + i * stride;
            uint2 *to = reinterpret_cast<uint2 *>(dst + i * stride * d);
            uint2 c = make_uint2(0, 0);
            if (row >= lo && row < hi) {
                float f[8];
                unpack8<T>(raw[i], f);
                c.x = C::encode4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
                c.y = C::encode4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
                *to = c;
            } else if (live && row < lo && (scale > old || mean)) {
                c = *to;
                if (scale > old) {  // old codes at the new scale
                    const float r = old * inv;
                    float f[4], g[4];
                    decode4<C>(c.x, f);
                    decode4<C>(c.y, g);
                    c.x = C::encode4(f[0] * r, f[1] * r, f[2] * r, f[3] * r);
                    c.y = C::encode4(g[0] * r, g[1] * r, g[2] * r, g[3] * r);
                    *to = c;
                }
            }
            if (mean)
                sum.add(c, finite && lo == 0);
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
                atomicAdd(&sums[col + j], sum.sum(j));
        __syncthreads();
        const float unit = 1.f / (static_cast<float>(C::kUnit) * page);  // a power of two
        float top = 0.f;
        for (int c = threadIdx.x; c < d; c += blockDim.x)
            top = fmaxf(top, fabsf(static_cast<float>(sums[c]) * unit));
        top = __uint_as_float(block_max(__float_as_uint(top), red));
        const int e = int8_exp(top);
        for (int c = threadIdx.x; c < d; c += blockDim.x)
            cache.k_mean[ph * d + c] = static_cast<int8_t>(scale_round(sums[c], C::kLog2Unit + cache.log2_page + e));
        if (threadIdx.x == 0)
            cache.k_mean_scale[ph] = pow2f(e) * scale;
    }
}

// No more new rows than sequences, as in a decoding step: one warp per (sequence,
// head, K or V), page by page; lane l holds columns 4 l .. 4 l + 3.  The same
// arithmetic; with a row or two a page nothing is worth holding, so a page's new
// rows are read once for amax and again to be encoded.  What it costs is the chain
// length - page number - scale and row, so the warps of a block share nothing and
// meet nowhere: one token of 8 heads takes 2.3 us against 3.3 with a block a page,
// 256 tokens (pages of 16) 6.7 against 7.2.  Where a token is larger than its page
// holds, the page's codes are read, moved to the new scale and written: 256 tokens of
// 8 heads into pages of 64 with 40 tokens in them take 3.2 us where the scales stay,
// 11 (e4m3) or 16 us (int8) where all of them grow.
constexpr int kStepWarps = 8;

template <typename T, typename C>
__global__ void __launch_bounds__(32 * kStepWarps) fa_cache_step_kernel(Cache cache, Batch batch, NewRows in, int d)
{
    const int lane = threadIdx.x & 31;
    const unsigned unit = blockIdx.x * kStepWarps + (threadIdx.x >> 5);
    const int which = unit & 1, h = static_cast<int>(unit / 2 % cache.heads), b = static_cast<int>(unit / 2 / cache.heads);
    if (b >= in.batch)
        return;
    const bool live = 4 * lane < d;
    const uint32_t infinity = DTypeTraits<T>::kBF16 ? 0x7F80u : 0x7C00u;
    const long long had = batch.seq_lens[b];  // tokens before
    int t0, n;
    if (!in.tokens(b, t0, n) || (n > 0 && had < 0)) {
        if (lane == 0)
            batch.bad();
        return;
    }
    if (n == 0)
        return;
    const long long end = had + n, last = (end - 1) >> cache.log2_page;
    const int page = cache.page;
    const long long token_stride = which ? in.token_stride[1] : in.token_stride[0];
    const T *x = static_cast<const T *>(which ? in.x[1] : in.x[0]) +
                 h * (which ? in.head_stride[1] : in.head_stride[0]) + 4 * lane;
    uint8_t *codes = which ? cache.v : cache.k;
    float *scales = which ? cache.v_scale : cache.k_scale;
    for (long long at = had >> cache.log2_page; at <= last; ++at) {
        const int p = at < batch.max_pages ? batch.page(b, static_cast<int>(at)) : -1;
        const long long base = at << cache.log2_page;  // position of the page's slot 0
        const int lo = static_cast<int>(max(had - base, 0ll));
        const int hi = static_cast<int>(min(end - base, static_cast<long long>(page)));
        const T *src = x + (t0 + (base - had)) * token_stride;  // of slot 0, if that is new
        auto row_of = [&](int row) -> uint2 {
            return live ? *reinterpret_cast<const uint2 *>(src + row * token_stride) : make_uint2(0, 0);
        };
        uint32_t m = 0;  // the rows are on their way while the page number is
#pragma unroll 4
        for (int row = lo; row < hi; ++row) {
            const uint2 r = row_of(row);
            m = max_magnitude2<T>(m, max_magnitude2<T>(r.x, r.y));
        }
        if (p < 0) {
            if (lane == 0)
                batch.bad();
            continue;
        }
        const size_t ph = static_cast<size_t>(p) * cache.heads + h;
        const float old = lo > 0 ? scales[ph] : 0.f;
        m &= 0x7FFF7FFFu;
        m = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
        float a = DTypeTraits<T>::unpack(m).x;
        if (m >= infinity) {  // the largest of the finite ones
            a = 0.f;
            for (int row = lo; row < hi; ++row) {
                const uint2 r = row_of(row);
                const float2 y = DTypeTraits<T>::unpack(r.x), z = DTypeTraits<T>::unpack(r.y);
                const float f[8] = {y.x, y.y, z.x, z.y, 0.f, 0.f, 0.f, 0.f};
                a = finite_max(a, f);
            }
            a = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
        }
        const float scale = fmaxf(old, pow2f(C::exp_of(a)));
        const float inv = 1.f / scale;
        uint8_t *dst = codes + ph * page * d + 4 * lane;
        const bool mean = which == 0 && hi == page && cache.k_mean != nullptr;
        int sum[4] = {0, 0, 0, 0};
        auto add = [&](uint32_t c) {
            float f[4];
            decode4<C>(c, f);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sum[j] += __float2int_rn(f[j] * C::kUnit);  // NaN converts to 0
        };
        if (live && (scale > old || mean)) {
#pragma unroll 16
            for (int row = 0; row < lo; ++row) {
                uint32_t *to = reinterpret_cast<uint32_t *>(dst + row * d);
                uint32_t c = *to;
                if (scale > old) {  // old codes at the new scale
                    const float r = old * inv;
                    float f[4];
                    decode4<C>(c, f);
                    c = C::encode4(f[0] * r, f[1] * r, f[2] * r, f[3] * r);
                    *to = c;
                }
                if (mean)
                    add(c);
            }
        }
        if (live) {
#pragma unroll 4
            for (int row = lo; row < hi; ++row) {
                const uint2 r = row_of(row);
                const float2 y = DTypeTraits<T>::unpack(r.x), z = DTypeTraits<T>::unpack(r.y);
                const uint32_t c = C::encode4(y.x * inv, y.y * inv, z.x * inv, z.y * inv);
                *reinterpret_cast<uint32_t *>(dst + row * d) = c;
                if (mean)
                    add(c);
            }
        }
        if (lane == 0)
            scales[ph] = scale;
        if (mean) {
            const float per = 1.f / (static_cast<float>(C::kUnit) * page);  // a power of two
            float top = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                top = fmaxf(top, fabsf(static_cast<float>(sum[j]) * per));
            top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
            const int e = int8_exp(top);
            uint32_t r = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                r |= static_cast<uint32_t>(scale_round(sum[j], C::kLog2Unit + cache.log2_page + e) & 0xFF) << (8 * j);
            if (live)
                *reinterpret_cast<uint32_t *>(cache.k_mean + ph * d + 4 * lane) = r;
            if (lane == 0)
                cache.k_mean_scale[ph] = pow2f(e) * scale;
        }
    }
}

// ---------------------------------------------------------------------------
// Reading back
//
// 16 codes (16 bytes) in, 16 values (32 bytes) out a thread and step; bound by
// the bytes it writes.  Two steps a thread: 8 x 16,384 tokens of 8 heads of 128
// (749 MB) take 116 us on the GPU, 95 % of the measured copy rate; one step 137, four 127,
// eight 151, and 8 codes a step 153 us.
constexpr int kReadThreads = 256;
constexpr int kReadSteps = 2;

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
    if (chunk == 0 && h == 0 && which == 0 && threadIdx.x == 0)
        batch.check_length(b, cache.log2_page);
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

// Scores of 128 pages of one (sequence, KV head) a block, for every query: int8
// products on the tensor cores (m16n8k32, int32 sums), 16 pages a warp as the
// rows, eight query heads as the columns.  The order of d in the product is
// free: a lane holds D / 4 consecutive bytes of two pages' means, loaded
// straight into the operand, and the same bytes of a query row from shared
// memory.  Query heads are padded to eights, query by query; a padded row's
// scale is NaN, which fmaxf passes over.  d + 4 bytes a page are read once; what
// the kernel costs is the latency of length, page number, mean and query row,
// so the first three are under way while the rows are rounded to int8.  With the
// choice below: 9.8 us for one sequence of 2,048 pages and 8 heads, 24 us for 32 of
// up to 2,048 pages, 4 heads and 2 queries (17 MB of means), of which the scores are the
// larger part (cold and alone 17 us against 12 for the choice): each of its 2,048 blocks
// goes through that chain and rounds the same query rows again.
constexpr int kScoreThreads = 256;
constexpr int kScorePages = kScoreThreads / 32 * 16;
constexpr int kScoreRows = 64;  // of shared memory at a time

__device__ __forceinline__ void mma_s8(int (&d)[4], int a0, int a1, int a2, int a3, int b0, int b1)
{
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int D, typename T>
__global__ void __launch_bounds__(kScoreThreads)
    fa_cache_score_kernel(Cache cache, Batch batch, Queries q, uint32_t *__restrict__ scores, int slots)
{
    constexpr int QUARTER = D / 16;  // 32-bit words a lane, page and row
    constexpr int STRIDE = D / 4 + 4;  // words of a row in shared memory
    __shared__ __align__(16) int q8[kScoreRows][STRIDE];
    __shared__ float q8_scale[kScoreRows];
    wait_ahead();
    let_next();
    const int b = blockIdx.z, h = blockIdx.y;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int first = (blockIdx.x * (kScoreThreads / 32) + warp) * 16;
    int page[2];  // of pages first + g, + 8; read before the length is known
#pragma unroll
    for (int x = 0; x < 2; ++x)
        page[x] = batch.page(b, first + g + 8 * x);
    const int len = batch.length(b, cache.log2_page);
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0)
        batch.check_length(b, cache.log2_page);
    const int n = (context(q, len, q.Nq - 1) + cache.page - 1) >> cache.log2_page;  // of the longest context
    if (static_cast<int>(blockIdx.x) * kScorePages >= n || n <= slots)
        return;  // no page here, or every page is chosen anyway
    int mean[2][QUARTER];
    float mean_scale[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        // a page that is not complete has no summary yet; it is the last of
        // every context that reaches it
        const bool whole = first + g + 8 * x < (len >> cache.log2_page);
        if (whole && page[x] < 0)
            batch.bad();
        if (!whole)
            page[x] = -1;
        mean_scale[x] = 0.f;
#pragma unroll
        for (int i = 0; i < QUARTER; ++i)
            mean[x][i] = 0;
        if (page[x] >= 0) {
            const size_t ph = static_cast<size_t>(page[x]) * cache.heads + h;
            mean_scale[x] = cache.k_mean_scale[ph];
            const int2 *src = reinterpret_cast<const int2 *>(cache.k_mean + ph * D) + c * (QUARTER / 2);
#pragma unroll
            for (int i = 0; i < QUARTER / 2; ++i) {
                const int2 w = src[i];
                mean[x][2 * i] = w.x;
                mean[x][2 * i + 1] = w.y;
            }
        }
    }
    const int tiles = (q.G + 7) / 8;  // of one query's heads
    const int all_rows = q.Nq * tiles * 8;
    float best[2] = {0.f, 0.f};
    for (int r0 = 0; r0 < all_rows; r0 += kScoreRows) {
        const int rows = min(kScoreRows, all_rows - r0);
        __syncthreads();  // the rows before are read
        for (int r = warp; r < rows; r += kScoreThreads / 32) {
            const int i = (r0 + r) / (tiles * 8), head = (r0 + r) % (tiles * 8);
            // lane l holds columns 4 l .. 4 l + 3
            float f[4] = {0.f, 0.f, 0.f, 0.f};
            if (head < q.G && lane < D / 4) {
                const T *src = static_cast<const T *>(q.q) + b * q.batch_stride +
                               static_cast<long long>(h * q.G + head) * q.head_stride + i * q.row_stride;
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
                q8[r][lane] = static_cast<int>(I8::encode4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv));
            if (lane == 0)
                q8_scale[r] = head < q.G ? pow2f(e) : __int_as_float(0x7FC00000);
        }
        __syncthreads();
        for (int r = 0; r < rows; r += 8) {
            int dot[4] = {0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < QUARTER; s += 2) {
                const int2 y = *reinterpret_cast<const int2 *>(&q8[r + g][c * QUARTER + s]);
                mma_s8(dot, mean[0][s], mean[1][s], mean[0][s + 1], mean[1][s + 1], y.x, y.y);
            }
            const int tile = (r0 + r) / 8 % tiles;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                // whole numbers below 2^21, and powers of two: exact
                const float s0 = (static_cast<float>(dot[2 * x]) * q8_scale[r + 2 * c]) * mean_scale[x];
                const float s1 = (static_cast<float>(dot[2 * x + 1]) * q8_scale[r + 2 * c + 1]) * mean_scale[x];
                const float top = fmaxf(s0, s1);
                best[x] = tile == 0 ? top : fmaxf(best[x], top);
            }
            if (tile == tiles - 1) {  // the query's last heads
                const long long seg = (static_cast<long long>(b) * cache.heads + h) * q.Nq + (r0 + r) / (tiles * 8);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float top = fmaxf(best[x], __shfl_xor_sync(0xffffffffu, best[x], 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const int at = first + g + 8 * x;
                    if (c == 0 && at < n)
                        scores[seg * batch.max_pages + at] = page[x] >= 0 ? ordered(top) : 0u;
                }
            }
        }
    }
}

// The `want` largest of the candidates' scores, ties to the lower page, with
// the kept pages, in ascending order.  One block a (sequence, KV head, query):
// the smallest chosen score by four 8-bit digits (a histogram of the scores
// that share the digits found so far), then one ordered pass that writes, each
// thread a run of pages.  Up to kPickHeld scores are held in shared memory.
//
// A table of at most kPickFew pages gives a block no more than two scores a
// thread with 128 threads, and 16 such blocks share an SM instead of four: the
// selection takes 18.5 us instead of 35.5 for 77 sequences x 8 heads x 4 queries
// of 26 pages, 9.9 instead of 12.5 for 39 x 32 of 133, 8.4 instead of 9.0 for
// 7 x 8 x 2 of 214, and 7.8 instead of 7.7 for 6 x 8 of 177.  A warp a segment,
// with its scores in registers and ballots for counts, took twice as long (19.5
// at 7 x 8 x 2 of 214).  Over 256 pages 512 threads stay: 256 threads took 10.5
// instead of 9.8 at 8 segments of 2,048 pages.
constexpr int kPickThreads = 512, kPickHeld = 8192;
constexpr int kPickFewThreads = 128, kPickFew = 256;

// Sum over the block's earlier threads of x (and, in `total`, over all).
template <int THREADS>
__device__ __forceinline__ int block_before(int x, int *smem, int &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off)
            incl += y;
    }
    __syncthreads();  // earlier reads of smem are done
    if (lane == 31)
        smem[warp] = incl;
    __syncthreads();
    total = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        const int y = smem[w];
        if (w < warp)
            incl += y;
        total += y;
    }
    return incl - x;
}

template <int THREADS, int HELD>
__global__ void __launch_bounds__(THREADS)
    fa_cache_pick_kernel(Cache cache, Batch batch, Queries q, const uint32_t *__restrict__ scores,
                         int *__restrict__ pages, int slots, int keep_first, int keep_last)
{
    __shared__ uint32_t held[HELD];
    __shared__ int hist[256];
    __shared__ int sums[THREADS / 32];
    __shared__ int found[2];
    wait_ahead();
    let_next();
    const long long seg = blockIdx.x;
    const int i = static_cast<int>(seg % q.Nq);
    const int b = static_cast<int>(seg / q.Nq / cache.heads);
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    int *out = pages + seg * slots;
    const int n = (context(q, batch.length(b, cache.log2_page), i) + cache.page - 1) >> cache.log2_page;
    if (n <= slots) {
        for (int j = t; j < slots; j += THREADS)
            out[j] = j < n ? j : -1;
        return;
    }
    const uint32_t *key = scores + seg * batch.max_pages;
    const int lo = keep_first, hi = n - keep_last;  // candidates
    const bool any = slots > keep_first + keep_last;
    int want = slots - keep_first - keep_last;      // < hi - lo
    if (n <= HELD && any) {
        for (int j = lo + t; j < hi; j += THREADS)
            held[j] = key[j];
        key = held;
    }
    uint32_t prefix = 0;
    for (int shift = 24; want > 0 && shift >= 0; shift -= 8) {
        for (int digit = t; digit < 256; digit += THREADS)
            hist[digit] = 0;
        __syncthreads();
        for (int j0 = lo; j0 < hi; j0 += THREADS) {
            const int j = j0 + t;
            const uint32_t x = j < hi ? key[j] : 0u;
            const bool in = j < hi && (shift == 24 || (x >> (shift + 8)) == prefix);
            const unsigned digit = in ? (x >> shift) & 255u : 256u;
            if (shift == 24) {  // few different ones: one addition for the lanes of a digit
                const unsigned same = __match_any_sync(0xffffffffu, digit);
                if (in && lane == __ffs(same) - 1)
                    atomicAdd(&hist[digit], __popc(same));
            } else if (in) {
                atomicAdd(&hist[digit], 1);
            }
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
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    if (before < want && before + c[u] >= want) {
                        found[0] = 255 - 8 * lane - u;
                        found[1] = want - before;
                    }
                    before += c[u];
                }
            }
        }
        __syncthreads();
        prefix = (prefix << 8) | static_cast<uint32_t>(found[0]);
        want = found[1];  // still to take among the scores that begin with `prefix`
    }
    // a page is written if it is kept, above the smallest chosen score, or one of
    // the first `want` that equal it
    const int each = (n + THREADS - 1) / THREADS;
    const int j0 = t * each, j1 = min(n, j0 + each);
    int above = 0, equal = 0, total;
    for (int j = j0; j < j1; ++j) {
        const bool kept = j < lo || j >= hi;
        const uint32_t x = !kept && any ? key[j] : 0u;
        above += kept || (any && x > prefix);
        equal += !kept && any && x == prefix;
    }
    const int equal_before = block_before<THREADS>(equal, sums, total);
    const int take = max(0, min(equal, want - equal_before));  // of its equal ones
    int pos = block_before<THREADS>(above + take, sums, total), left = take;
    for (int j = j0; j < j1; ++j) {
        const bool kept = j < lo || j >= hi;
        const uint32_t x = !kept && any ? key[j] : 0u;
        bool in = kept || (any && x > prefix);
        if (!in && any && x == prefix && left > 0) {
            --left;
            in = true;
        }
        if (in)
            out[pos++] = j;
    }
}

}  // namespace cache
}  // namespace fa
