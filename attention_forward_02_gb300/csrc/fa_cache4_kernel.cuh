// fa_cache4_kernel.cuh -- the 4-bit paged KV cache on sm_103a: writing rows into
// its slots and reading sequences back.  The attention over it is in
// fa_cache4_decode_kernel.cuh, fa_cache4_short_kernel.cuh and fa_cache4_tc_kernel.cuh.
//
// Sixteen channels of a token share a scale of 5 exponent and 3 fraction bits; the
// byte is bits 14 .. 7 of an fp16, so that a shift decodes it.  Codes are e2m1, which
// the hardware converts.  Their product has at most 2 x 4 significant bits and the
// lowest is 2^-18: exact in fp16 and in bf16.
//
// A page and head is one block of bytes, [K codes | K scales | V codes | V scales], so
// that one copy fetches a page for attention.
#pragma once

#include "fa_cache_kernel.cuh"

namespace fa {
namespace cache4 {

using cache::Batch;

constexpr int kGroup = 16;           // channels a scale
constexpr float kTopScale = 10240.f;  // 6 of it fit fp16

struct Cache4 {
    uint8_t *data;
    int num_pages, heads, page, log2_page;
};

// Bytes of K (or V) of a page and head.
__host__ __device__ __forceinline__ int half_block(int page, int d) { return page * d / 16 * 9; }

__device__ __forceinline__ uint32_t load_u8(uint32_t addr)
{
    uint32_t x = 0;
    if (smem_ok(addr, 1, 1))
        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(x) : "r"(addr) : "memory");
    return x;
}
__device__ __forceinline__ uint32_t load_u16(uint32_t addr)
{
    uint32_t x = 0;
    if (smem_ok(addr, 2, 2))
        asm volatile("ld.shared.u16 %0, [%1];" : "=r"(x) : "r"(addr) : "memory");
    return x;
}

// A scale byte's value, in both halves of a pair.
__device__ __forceinline__ uint32_t scale_pair(uint32_t byte) { return (byte << 7) | (byte << 23); }

// Eight codes to four pairs of fp16, channels 2 i and 2 i + 1 in h[i].
__device__ __forceinline__ void halves8(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=&r"(h[0]), "=&r"(h[1]), "=&r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Codes of eight values (neighbours in pairs), the first in the lowest bits.
__device__ __forceinline__ uint32_t encode8(const float2 (&x)[4])
{
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(x[0].x), "f"(x[0].y), "f"(x[1].x), "f"(x[1].y), "f"(x[2].x), "f"(x[2].y), "f"(x[3].x), "f"(x[3].y));
    return w;
}

// The scale of a block, amax / 6 rounded to the nearest (ties to even) 5-3 number.
// Both roundings: the quotient to fp32, then to a multiple of 2^(e-3), or 2^-17.  An
// 11-bit amax is either six times a tie, whose quotient is exact, or at least 2^-11 of it
// away, so that the first does not disturb the second.
__device__ __forceinline__ float scale_of(float amax)
{
    const float t = __fdiv_rn(amax, 6.f);
    const int e = max(static_cast<int>(__float_as_uint(t) >> 23), 127 - 14);
    const float c = __uint_as_float(static_cast<uint32_t>(e + 20) << 23 | 0x400000u);  // 1.5 2^(e+20): its ulp is 2^(e-3)
    return fminf(__fsub_rn(__fadd_rn(t, c), c), kTopScale);
}

// ---------------------------------------------------------------------------
// Writing
//
// A thread takes one block of 16 channels of a token's K and the same of its V: four
// 16-byte loads under way, eight code bytes and a scale byte out each.  Threads of a
// block: the token's blocks of channels, then tokens, of one head, so that the scale
// bytes of neighbouring slots leave a warp together.
//
// A quotient x / scale is rounded to the multiple of 2^-13 next to it, by adding 1536 to
// x times the scale's reciprocal in one fused operation and taking it off again.  The
// borders between codes are multiples of 2^-2, so that a quotient on one comes out as one
// although the reciprocal is rounded (6.4 2^-24 at most).  Any other keeps its side: with
// x = X 2^i, X < 2^11, and scale = S 2^j, S < 2^4, the quotient is off a border k / 4 by
// (4 X 2^i - k S 2^j) / (4 S 2^j), which for X > 100 is no less than 1 / 4 / X > 2^-13 (i < j - 1
// there, and both terms multiples of 4 2^i), and for a smaller X no less than 2^-11.
//
// 58,800 tokens of 8 heads of 128 (308 MB) take 50.8 us on the GPU from fp16, 89 % of the
// measured copy rate: 185 instructions a block of channels keep the schedulers 71 % busy, which
// leaves the loads too few; 32-byte loads change nothing.  256 tokens take 2.0 us.
constexpr int kWriteThreads = 256;

struct Rows4 {
    const void *x[2];  // K, V
    long long token_stride[2], head_stride[2];
    const int *slots;
    int total;
};

template <typename T>
__device__ __forceinline__ void write_block(const uint4 (&raw)[2], uint8_t *codes, uint8_t *scale_to)
{
    uint32_t w[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
    constexpr uint32_t infinity = DTypeTraits<T>::kBF16 ? 0x7F80u : 0x7C00u;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = cache::max_magnitude2<T>(m, w[i]);
    m &= 0x7FFF7FFFu;
    m = max(m & 0xFFFFu, m >> 16);
    if (m >= infinity) {  // the largest finite one; NaN becomes 0
        m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
            w[i] &= (lo > infinity ? 0u : 0xFFFFu) | (hi > infinity ? 0u : 0xFFFF0000u);
            m = max(m, max(lo < infinity ? lo : 0u, hi < infinity ? hi : 0u));
        }
    }
    const float scale = scale_of(DTypeTraits<T>::unpack(m).x);
    uint2 c = make_uint2(0, 0);
    if (scale > 0.f) {
        const float inv = __frcp_rn(scale);
        const float2 by = make_float2(inv, inv), up = make_float2(1536.f, 1536.f), down = make_float2(-1536.f, -1536.f);
        uint32_t code[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t *v = w + 4 * j;
            float2 f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[i] = fadd2(ffma2(DTypeTraits<T>::unpack(v[i]), by, up), down);
            // what became 0 on the way keeps its sign: the values' top bits, two bytes of each
            // word, to the codes' top bits
            const uint32_t x = __byte_perm(v[0], v[1], 0x7351), y = __byte_perm(v[2], v[3], 0x7351);
            code[j] = encode8(f) | ((__byte_perm(x, y, 0x5410) & 0x80808080u) >> 4) | (__byte_perm(x, y, 0x7632) & 0x80808080u);
        }
        c = make_uint2(code[0], code[1]);
    }
    *reinterpret_cast<uint2 *>(codes) = c;
    *scale_to = static_cast<uint8_t>(__half_as_ushort(__float2half_rn(scale)) >> 7);
}

template <typename T>
__global__ void __launch_bounds__(kWriteThreads) fa_cache4_write_kernel(Cache4 cache, Rows4 in, int d, unsigned int *status)
{
    cache::wait_ahead();
    cache::let_next();
    const int groups = d / kGroup;
    const int tokens = kWriteThreads / groups;
    const int lane = threadIdx.x / groups, g = threadIdx.x % groups;
    const long long t = static_cast<long long>(blockIdx.x) * tokens + lane;
    const int h = blockIdx.y;
    if (lane >= tokens || t >= in.total)
        return;
    const int slot = in.slots[t];
    uint4 raw[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const T *src = static_cast<const T *>(in.x[i]) + t * in.token_stride[i] + h * in.head_stride[i] + g * kGroup;
        raw[i][0] = *reinterpret_cast<const uint4 *>(src);
        raw[i][1] = *reinterpret_cast<const uint4 *>(src + 8);
    }
    if (slot < 0)
        return;
    const int p = slot >> cache.log2_page, row = slot & (cache.page - 1);
    if (p >= cache.num_pages) {
        atomicOr(status, kStatusBounds);
        return;
    }
    const int half = half_block(cache.page, d);
    uint8_t *block = cache.data + (static_cast<size_t>(p) * cache.heads + h) * (2 * half);
#pragma unroll
    for (int i = 0; i < 2; ++i, block += half)
        write_block<T>(raw[i], block + row * (d / 2) + g * 8, block + cache.page * (d / 2) + row * groups + g);
}

// ---------------------------------------------------------------------------
// Reading back
//
// A block of 16 channels (8 code bytes, a scale byte) in, 32 bytes out a thread and
// step; bound by the bytes it writes, so that they leave in one 32-byte store, a whole
// sector (two of 16 bytes, which leave a warp in half sectors, take 8 x 16,384 tokens of 8
// heads of 128, 656 MB, from 98.5 to 117.7 us on the GPU; outputs on odd 16 bytes have
// them).  98 % of the measured copy rate; four steps a thread 98.8 us.
constexpr int kReadThreads = 256;
constexpr int kReadSteps = 2;

template <typename T>
__global__ void __launch_bounds__(kReadThreads)
    fa_cache4_read_kernel(Cache4 cache, Batch batch, T *__restrict__ k, T *__restrict__ v, int N, int d, int chunks)
{
    // blockIdx.x = (b * heads + h) * chunks + chunk; y: K or V
    cache::wait_ahead();
    cache::let_next();
    const int which = blockIdx.y;
    const long long bh = blockIdx.x / chunks;
    const int chunk = blockIdx.x % chunks;
    const int b = static_cast<int>(bh / cache.heads), h = static_cast<int>(bh % cache.heads);
    const int groups = d / kGroup;
    const long long vectors = static_cast<long long>(N) * groups;
    const int len = batch.length(b, cache.log2_page);
    if (chunk == 0 && h == 0 && which == 0 && threadIdx.x == 0)
        batch.check_length(b, cache.log2_page);
    T *out = (which ? v : k) + bh * N * d;
    const bool whole = (reinterpret_cast<uintptr_t>(out) & 31) == 0;  // d is a multiple of 16 values: every block is then
    const int half = half_block(cache.page, d);
    const long long first = static_cast<long long>(chunk) * (kReadThreads * kReadSteps) + threadIdx.x;
    uint2 c[kReadSteps];
    uint32_t s[kReadSteps];
#pragma unroll
    for (int i = 0; i < kReadSteps; ++i) {
        const long long at = first + i * kReadThreads;
        c[i] = make_uint2(0, 0);
        s[i] = 0;
        const int t = static_cast<int>(at / groups), g = static_cast<int>(at % groups);
        if (at < vectors && t < len) {
            const int p = batch.page(b, t >> cache.log2_page);
            if (p >= 0) {
                const uint8_t *block = cache.data + (static_cast<size_t>(p) * cache.heads + h) * (2 * half) + which * half;
                const int row = t & (cache.page - 1);
                c[i] = *reinterpret_cast<const uint2 *>(block + row * (d / 2) + g * 8);
                s[i] = block[cache.page * (d / 2) + row * groups + g];
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
        uint32_t h8[2][4], r[8];
        halves8(c[i].x, h8[0]);
        halves8(c[i].y, h8[1]);
        const uint32_t by = scale_pair(s[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const __half2 x = __hmul2(*reinterpret_cast<const __half2 *>(&h8[j >> 2][j & 3]),
                                      *reinterpret_cast<const __half2 *>(&by));  // exact
            if (DTypeTraits<T>::kBF16) {
                const float2 y = __half22float2(x);
                r[j] = DTypeTraits<T>::pack(y.x, y.y);
            } else {
                r[j] = *reinterpret_cast<const uint32_t *>(&x);
            }
        }
        uint4 *dst = reinterpret_cast<uint4 *>(out + at * kGroup);
        if (whole) {
            asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(r[0]), "r"(r[1]),
                         "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                         : "memory");
        } else {
            __stcs(dst, make_uint4(r[0], r[1], r[2], r[3]));
            __stcs(dst + 1, make_uint4(r[4], r[5], r[6], r[7]));
        }
    }
}

}  // namespace cache4
}  // namespace fa
