// fa_cache4.cu -- host side of the 4-bit paged KV cache declared in include/fa.h:
// argument checks and the launches of writing, reading back and decoding attention.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <functional>
#include <mutex>

#include "fa.h"
#include "fa_cache4_decode_kernel.cuh"
#include "fa_cache4_kernel.cuh"
#include "fa_cache4_short_kernel.cuh"
#include "fa_cache4_tc_kernel.cuh"
#include "fa_cache_host.h"
#include "fa_host.h"

namespace {

using namespace fa_host;
using fa::cache4::Batch;
using fa::cache4::Cache4;

struct Cache4State {
    std::once_flag once;
    cudaError_t err = cudaErrorUnknown;
    unsigned int *status = nullptr;
};
Cache4State g_cache4[kMaxDevices];

// Units of 128 keys of a segment that one block may take whole: one launch in place of two,
// but the units one after the other.  8 KV heads of 4 rows, whole / shared out, us on the
// GPU (in a graph):
//                      1 unit       4 units      8 units      12 units
//   d = 128, 1 seq.    4.1 / 6.5    6.2 / 8.6    9.1 / 8.7    12.1 / 8.8
//            16        4.4 / 6.8    6.6 / 9.9    9.7 / 11.0   13.0 / 11.5
//            56        6.0 / 8.2    10.1 / 14.5  15.2 / 17.8  20.4 / 21.0
//   d = 64,  1         3.5 / 5.7    5.2 / 7.5    7.3 / 7.5    9.6 / 7.8
//            56        4.4 / 6.8    6.8 / 10.7   10.1 / 12.7  14.2 / 15.6
//   d = 32,  16        3.6 / 5.8    5.1 / 7.9    7.2 / 8.1    9.3 / 8.3
constexpr long long kWholeUnits = 8;

// More segments than resident blocks go to a warp each where they are bounded to this many
// units, one more for every segment a block, kWholeUnits at most.  Up to 8 rows; a warp each /
// shared out, us on the GPU (in a graph), contexts of up to
//                                   1 unit        3 units        4 units        6 units        8 units
//   d = 128,   512 segments, 4 rows 6.3 / 10.5    13.4 / 13.7    16.9 / 13.9    24.1 / 17.5    31.2 / 18.9
//             1024                  7.7 / 15.0    16.4 / 20.6    20.7 / 22.1    29.2 / 25.1    38.1 / 27.8
//             2048                  11.7 / 24.4   23.8 / 32.1    30.3 / 36.0    42.6 / 41.3    54.2 / 48.7
//             4096                  18.6 / 41.3   36.7 / 56.5    46.7 / 63.7    64.4 / 76.1    78.0 / 85.0
//                          8 rows   20.8 / 51.0   40.3 / 68.4    51.3 / 76.1    71.2 / 90.1    86.1 / 100
//   d = 64,    512           1 row  5.2 / 8.3     10.8 / 10.5    13.8 / 11.3    19.4 / 12.4    25.2 / 13.8
//             4096                  12.8 / 26.0   25.4 / 37.2    32.2 / 40.8    43.5 / 50.0    56.4 / 57.0
//   d = 32,   1024           4 rows 5.3 / 9.8     11.1 / 13.1    13.8 / 13.7    19.6 / 15.4    25.4 / 17.4
// With no more segments than blocks a block each is ahead from 2 units on: 384 of up to 300
// keys 8.1 where a warp each takes 11.4.
constexpr long long kShortUnits = 2;

// More than 16 rows (d = 128; 32 at d = 96): the tcgen05 kernel has one block an SM, to which a
// segment's begin and end cost about five units of 128 keys, so that batches of short segments are
// faster with the other one, two blocks an SM of which each takes a segment whole.  tcgen05 / the other, us
// on the GPU (in a graph), contexts of up to
//                                      1 unit       2            3            4            5            6            8
//   d = 128, 24 rows,   64 segments    8.2 / 8.5    9.5 / 9.9                 11.3 / 13.0                            15.6 / 19.7
//                      160             16.0 / 9.6   16.1 / 11.7  18.3 / 14.1  19.6 / 15.8  20.1 / 18.0  20.8 / 21.4  23.6 / 25.3
//                      304             17.5 / 10.3  22.0 / 12.3  25.1 / 14.8  26.4 / 17.2  26.1 / 19.3  28.2 / 21.9  31.1 / 27.0
//                     1024             46.9 / 40.7  53.7 / 48.2  58.5 / 49.7  62.5 / 58.6  65.4 / 63.5  68.6 / 69.0  76.5 / 78.8
//                     2048             88.1 / 69.2  98.3 / 83.5  104 / 90.8   111 / 101    117 / 110    127 / 120    142 / 141
//            64 rows,   64             10.1 / 12.3  11.7 / 15.0               14.6 / 21.3                            20.9 / 34.2
//                      160             22.7 / 14.1  22.7 / 18.2  25.6 / 22.6  26.7 / 27.1  27.6 / 30.5  29.5 / 37.5  33.0 / 45.4
//                      304             25.5 / 15.6  32.0 / 19.5  37.0 / 24.7  37.7 / 28.2  38.1 / 33.5  41.2 / 38.4  44.9 / 47.4
//                     1024             73.4 / 73.2  82.8 / 88.5  89.4 / 90.8  95.1 / 104   99.8 / 117
//                     2048             145 / 132    158 / 159    166 / 172    177 / 190    187 / 209
//   d = 96,  64 rows,   64             10.1 / 10.0  12.0 / 13.0               14.0 / 18.5                            20.1 / 30.2
//            36 rows,   64             9.9 / 8.7    11.3 / 11.9               14.1 / 17.4                            19.5 / 29.1
//                      160             20.6 / 10.1  20.8 / 13.8  23.0 / 17.5  25.0 / 21.4  25.0 / 24.3  26.6 / 30.2  29.9 / 37.0
//                      304             22.7 / 10.8  28.8 / 15.0  33.4 / 18.5  34.6 / 22.3  34.6 / 26.1  37.2 / 31.2  40.4 / 39.1
//                     2048             120 / 84.9   133 / 104    141 / 120    151 / 137    160 / 148    171 / 172    189 / 200
// At d = 96 it is also behind where few units are shared out: 8 segments of 10, 16, 32, 64 units
// 19.5 / 17.4, 20.0 / 17.9, 20.8 / 18.7, 21.5 / 22.6, 16 of 16 and 24 units 20.2 / 18.6, 20.6 / 21.9 (at d = 128 8 of 16
// units, 17 rows 16.5 / 15.4, 32 rows 17.1 / 16.4, 64 rows 21.3 / 23.7).
template <int D>
bool on_tcgen05(int rows, long long segments, long long units, int sms)
{
    const bool more = segments > sms;
    if (D == 96)
        return rows > 32 && units > (more ? 5 : 1) && (units <= kWholeUnits || segments * units > 256);
    if (rows <= 32)
        return rows > 16 && units > (more ? 8 : 0);
    return units > (!more ? 0 : segments <= 2 * sms ? 4 : 2);
}

template <int D, int ROWS, typename T>
constexpr auto decode_kernel()
{
    return fa::cache4::fa_cache4_decode_kernel<D, ROWS, T>;
}

template <int D, int ROWS>
cudaError_t set_smem_attr()
{
    const cudaFuncAttribute a = cudaFuncAttributeMaxDynamicSharedMemorySize;
    constexpr int bytes = fa::cache4::Dec4Cfg<D, ROWS>::SMEM;
    cudaError_t e = cudaFuncSetAttribute(decode_kernel<D, ROWS, __half>(), a, bytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(decode_kernel<D, ROWS, __nv_bfloat16>(), a, bytes);
    if constexpr (ROWS <= 8) {
        constexpr int own = fa::cache4::Short4Cfg<D, ROWS>::SMEM;
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(fa::cache4::fa_cache4_short_kernel<D, ROWS, __half>, a, own);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(fa::cache4::fa_cache4_short_kernel<D, ROWS, __nv_bfloat16>, a, own);
    }
    return e;
}
template <int D, int ROWS>
cudaError_t set_tc_smem_attr()
{
    const cudaFuncAttribute a = cudaFuncAttributeMaxDynamicSharedMemorySize;
    constexpr int bytes = fa::cache4::Tc4Cfg<D, ROWS>::SMEM;
    const cudaError_t e = cudaFuncSetAttribute(fa::cache4::fa_cache4_tc_kernel<D, ROWS, __half>, a, bytes);
    return e == cudaSuccess ? cudaFuncSetAttribute(fa::cache4::fa_cache4_tc_kernel<D, ROWS, __nv_bfloat16>, a, bytes) : e;
}
template <int D>
cudaError_t set_smem_attrs()
{
    cudaError_t e = set_smem_attr<D, 4>();
    if (e == cudaSuccess)
        e = set_smem_attr<D, 8>();
    return e == cudaSuccess ? set_smem_attr<D, 16>() : e;
}

void init_cache4(Cache4State &st)
{
    void *p = nullptr;
    st.err = cudaGetSymbolAddress(&p, fa::g_fa_status);
    st.status = static_cast<unsigned int *>(p);
    if (st.err == cudaSuccess) st.err = set_smem_attrs<32>();
    if (st.err == cudaSuccess) st.err = set_smem_attrs<64>();
    if (st.err == cudaSuccess) st.err = set_smem_attrs<96>();
    if (st.err == cudaSuccess) st.err = set_smem_attrs<128>();
    if (st.err == cudaSuccess) st.err = set_tc_smem_attr<96, 64>();
    if (st.err == cudaSuccess) st.err = set_tc_smem_attr<128, 64>();
    if (st.err == cudaSuccess) st.err = set_tc_smem_attr<128, 32>();
}

// The current device's state and SM count.
fa_status_t device(Cache4State **out, int *num_sms)
{
    EncodeTiledFn encode = nullptr;
    const fa_status_t s = encoder(&encode, num_sms);
    if (s != FA_OK)
        return s;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        return FA_ERR_CUDA;
    Cache4State &st = g_cache4[dev];
    std::call_once(st.once, init_cache4, std::ref(st));
    if (st.err != cudaSuccess)
        return FA_ERR_CUDA;
    *out = &st;
    return FA_OK;
}

// Checks of a cache that need no device; its memory.
fa_status_t check_cache(const fa_cache4_t *c, Range *own)
{
    if (!c || c->num_pages < 1 || c->heads < 1)
        return FA_ERR_INVALID_ARG;
    if ((c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) ||
        (c->d != 32 && c->d != 64 && c->d != 96 && c->d != 128) || c->heads > kMaxBatch / 2 ||
        static_cast<long long>(c->num_pages) * c->heads > 0x7fffffffLL ||
        static_cast<long long>(c->num_pages) * c->page > 0x7fffffffLL)
        return FA_ERR_UNSUPPORTED;
    if (!c->data)
        return FA_ERR_INVALID_ARG;
    if (u(c->data) & 15u)
        return FA_ERR_MISALIGNED;
    *own = {u(c->data), static_cast<size_t>(c->num_pages) * c->heads * (2 * fa::cache4::half_block(c->page, c->d))};
    return FA_OK;
}

Cache4 device_cache(const fa_cache4_t *c)
{
    int log2_page = 4;
    while ((1 << log2_page) < c->page)
        ++log2_page;
    return {static_cast<uint8_t *>(c->data), c->num_pages, c->heads, c->page, log2_page};
}

template <typename F>
fa_status_t by_type(fa_dtype_t dtype, F f)
{
    return dtype == FA_FP16 ? f(__half()) : f(__nv_bfloat16());
}

// A warp for each of the segments, of up to eight rows.
template <int D, int ROWS>
fa_status_t launch_short(const fa::cache::Work &w, long long segments, void *o, float *lse, fa_dtype_t dtype, cudaStream_t cs)
{
    if constexpr (ROWS > 8) {
        return FA_ERR_UNSUPPORTED;
    } else {
        using S = fa::cache4::Short4Cfg<D, ROWS>;
        const unsigned blocks = static_cast<unsigned>((segments + S::WARPS - 1) / S::WARPS);
        return by_type(dtype, [&](auto t) {
            using T = decltype(t);
            return launch_dependent(fa::cache4::fa_cache4_short_kernel<D, ROWS, T>, blocks, S::THREADS, S::SMEM, cs, w,
                                    static_cast<T *>(o), lse)
                       ? launched()
                       : FA_ERR_CUDA;
        });
    }
}

}  // namespace

namespace fa_host {

unsigned int *cache4_status_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, fa::g_fa_status) == cudaSuccess ? static_cast<unsigned int *>(p) : nullptr;
}

}  // namespace fa_host

extern "C" {

fa_status_t fa_cache4_write(const fa_cache4_t *cache, const void *k, const void *v, long long k_token_stride,
                            long long k_head_stride, long long v_token_stride, long long v_head_stride,
                            const int *slots, int T, fa_dtype_t dtype, void *stream)
{
    Range own;
    fa_status_t s = check_cache(cache, &own);
    if (s != FA_OK)
        return s;
    if (T < 0)
        return FA_ERR_INVALID_ARG;
    if (dtype != FA_FP16 && dtype != FA_BF16)
        return FA_ERR_UNSUPPORTED;
    if (T == 0)
        return FA_OK;  // empty problem
    if (T == 1)        // the stride of a dimension of one means nothing
        k_token_stride = v_token_stride = 0;
    if (cache->heads == 1)
        k_head_stride = v_head_stride = 0;
    if (!k || !v || !slots || !fine(k_token_stride, T) || !fine(k_head_stride, cache->heads) || !fine(v_token_stride, T) ||
        !fine(v_head_stride, cache->heads))
        return FA_ERR_INVALID_ARG;
    if ((u(k) | u(v)) & 15u || u(slots) & 3u || !strides_aligned(k_token_stride, k_head_stride) ||
        !strides_aligned(v_token_stride, v_head_stride))
        return FA_ERR_MISALIGNED;
    const Range in[3] = {
        {u(k), static_cast<size_t>((T - 1) * k_token_stride + (cache->heads - 1) * k_head_stride + cache->d) * 2},
        {u(v), static_cast<size_t>((T - 1) * v_token_stride + (cache->heads - 1) * v_head_stride + cache->d) * 2},
        {u(slots), static_cast<size_t>(T) * 4}};
    if (any_overlap(own, in, 3))
        return FA_ERR_INVALID_ARG;
    Cache4State *st = nullptr;
    if ((s = device(&st, nullptr)) != FA_OK)
        return s;
    const fa::cache4::Rows4 rows = {
        {k, v}, {k_token_stride, v_token_stride}, {k_head_stride, v_head_stride}, slots, T};
    const int tokens = fa::cache4::kWriteThreads / (cache->d / fa::cache4::kGroup);
    const dim3 grid(static_cast<unsigned>((static_cast<long long>(T) + tokens - 1) / tokens), cache->heads);
    return by_type(dtype, [&](auto t) {
        return launch_dependent(fa::cache4::fa_cache4_write_kernel<decltype(t)>, grid, fa::cache4::kWriteThreads, 0,
                                static_cast<cudaStream_t>(stream), device_cache(cache), rows, cache->d, st->status)
                   ? launched()
                   : FA_ERR_CUDA;
    });
}

fa_status_t fa_cache4_read(const fa_cache4_t *cache, void *k, void *v, const int *seq_lens, const int *page_table,
                           long long table_stride, int max_pages, int B, int N, fa_dtype_t dtype, void *stream)
{
    Range own;
    fa_status_t s = check_cache(cache, &own);
    if (s != FA_OK)
        return s;
    if (B < 0 || N < 0)
        return FA_ERR_INVALID_ARG;
    if (dtype != FA_FP16 && dtype != FA_BF16)
        return FA_ERR_UNSUPPORTED;
    if (B == 0 || N == 0)
        return FA_OK;  // empty problem
    if ((s = check_batch(seq_lens, page_table, table_stride, max_pages, B, cache->page)) != FA_OK)
        return s;
    if (!k || !v)
        return FA_ERR_INVALID_ARG;
    if ((u(k) | u(v)) & 15u)
        return FA_ERR_MISALIGNED;
    constexpr int kPerBlock = fa::cache4::kReadThreads * fa::cache4::kReadSteps;
    const long long chunks = (static_cast<long long>(N) * (cache->d / fa::cache4::kGroup) + kPerBlock - 1) / kPerBlock;
    const long long blocks = chunks * B * cache->heads;
    if (blocks > 0x7fffffffLL)
        return FA_ERR_UNSUPPORTED;
    const size_t bytes = static_cast<size_t>(B) * cache->heads * N * cache->d * 2;
    const Range out[2] = {{u(k), bytes}, {u(v), bytes}};
    const Range in[3] = {own,
                         {u(seq_lens), static_cast<size_t>(B) * 4},
                         {u(page_table), (static_cast<size_t>(B - 1) * table_stride + max_pages) * 4}};
    if (any_overlap(out[0], in, 3) || any_overlap(out[1], in, 3) || any_overlap(out[0], out + 1, 1))
        return FA_ERR_INVALID_ARG;
    Cache4State *st = nullptr;
    if ((s = device(&st, nullptr)) != FA_OK)
        return s;
    const Batch batch = {seq_lens, page_table, table_stride, max_pages, cache->num_pages, st->status};
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        return launch_dependent(fa::cache4::fa_cache4_read_kernel<T>, dim3(static_cast<unsigned>(blocks), 2),
                                fa::cache4::kReadThreads, 0, static_cast<cudaStream_t>(stream), device_cache(cache), batch,
                                static_cast<T *>(k), static_cast<T *>(v), N, cache->d, static_cast<int>(chunks))
                   ? launched()
                   : FA_ERR_CUDA;
    });
}

size_t fa_decode_cache4_workspace_size(int B, int Hq, int Hkv, int Nq, int d)
{
    return fa_decode_cache_workspace_size(B, Hq, Hkv, Nq, d);
}

fa_status_t fa_decode_cache4(const fa_cache4_t *cache, const void *q, long long q_batch_stride, long long q_head_stride,
                             long long q_row_stride, void *o, float *lse, const int *seq_lens, const int *page_table,
                             long long table_stride, int max_pages, void *workspace, size_t workspace_bytes, int B, int Hq,
                             int Nq, float scale, int causal, fa_dtype_t dtype, void *stream)
{
    Range own;
    fa_status_t s = check_cache(cache, &own);
    if (s != FA_OK)
        return s;
    if (B < 0 || Hq < 0 || !std::isfinite(scale))
        return FA_ERR_INVALID_ARG;
    if (scale < 0.f)
        return FA_ERR_UNSUPPORTED;
    if (B == 0 || Hq == 0)
        return FA_OK;  // empty problem
    if ((s = check_batch(seq_lens, page_table, table_stride, max_pages, B, cache->page)) != FA_OK)
        return s;
    Range in[4] = {own};
    if ((s = check_queries(cache->heads, cache->d, q, q_batch_stride, q_head_stride, q_row_stride, B, Hq, Nq, causal, dtype,
                           in + 1)) != FA_OK)
        return s;
    const size_t need = fa_decode_cache4_workspace_size(B, Hq, cache->heads, Nq, cache->d);
    if (!o || !workspace || workspace_bytes < need)
        return FA_ERR_INVALID_ARG;
    if ((u(o) | u(workspace)) & 15u || u(lse) & 3u)
        return FA_ERR_MISALIGNED;
    const long long rows = static_cast<long long>(B) * Hq * Nq;
    if (rows > 0x7fffffffLL)
        return FA_ERR_UNSUPPORTED;
    in[2] = {u(seq_lens), static_cast<size_t>(B) * 4};
    in[3] = {u(page_table), (static_cast<size_t>(B - 1) * table_stride + max_pages) * 4};
    const Range out[3] = {{u(o), static_cast<size_t>(rows) * cache->d * 2},
                          {u(lse), static_cast<size_t>(rows) * 4},
                          {u(workspace), need}};
    for (int i = 0; i < 3; ++i)
        if (any_overlap(out[i], in, 4) || any_overlap(out[i], out, i))
            return FA_ERR_INVALID_ARG;
    Cache4State *st = nullptr;
    int sms = 0;
    if ((s = device(&st, &sms)) != FA_OK)
        return s;
    const Batch batch = {seq_lens, page_table, table_stride, max_pages, cache->num_pages, st->status};
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const Cache4 c = device_cache(cache);
    fa::cache::Work w = {};
    w.cache = {c.data, nullptr, nullptr, nullptr, nullptr, nullptr, c.num_pages, c.heads, c.page, c.log2_page};
    w.batch = batch;
    w.q = {q, q_batch_stride, q_head_stride, q_row_stride, Hq / cache->heads, Nq, causal};
    w.B = B;
    w.R = w.q.G * Nq;
    const Shape shape = shape_of(w.R);
    w.row_warps = shape.row_warps;
    const int rows_block = shape.rows_block;
    w.groups = (w.R + rows_block - 1) / rows_block;
    w.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    w.plan = static_cast<long long *>(workspace);
    const size_t part_rows = static_cast<size_t>(2 * fa::cache::kMaxBlocks) * rows_block;
    w.part_o = reinterpret_cast<float *>(static_cast<char *>(workspace) + plan_bytes(B));
    w.part_m = w.part_o + part_rows * cache->d;
    w.part_l = w.part_m + part_rows;
    const long long segments = static_cast<long long>(B) * cache->heads * w.groups;
    const long long bound = (static_cast<long long>(max_pages) * cache->page + 127) / 128;  // units of 128 keys
    return by_dim(cache->d, [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        // A kernel of F's runs: its grid, its launch, and the merge's.
        const auto run = [&](auto config, int per_sm, const auto &launch) {
            using F = decltype(config);
            const int box = cache->page < F::STEP ? cache->page : F::STEP;
            w.log2_box = box == 128 ? 7 : box == 64 ? 6 : box == 32 ? 5 : 4;
            const long long units = (static_cast<long long>(max_pages) * cache->page - 1) / F::STEP + 1;  // of one, at most
            long long blocks = std::min<long long>(static_cast<long long>(sms) * per_sm, fa::cache::kMaxBlocks);
            w.whole = bound <= kWholeUnits && segments <= blocks;
            blocks = w.whole ? segments : std::min(blocks, segments * units);
            return by_type(dtype, [&](auto t) {
                using T = decltype(t);
                if (!launch(t, static_cast<unsigned>(blocks)))
                    return FA_ERR_CUDA;
                if (w.whole)
                    return launched();
                constexpr int kWarps = fa::cache::kCombineThreads / 32;
                const bool second =
                    blocks <= segments * fa::cache::kCombineEach
                        ? launch_dependent(fa::cache::fa_cache_combine_kernel<D, T, 1, F::LOG2_STEP, F::OPEN>,
                                           static_cast<unsigned>((rows + kWarps - 1) / kWarps), fa::cache::kCombineThreads,
                                           0, cs, w, static_cast<T *>(o), lse, rows_block, rows)
                        : launch_dependent(fa::cache::fa_cache_combine_kernel<D, T, kWarps, F::LOG2_STEP, F::OPEN>,
                                           static_cast<unsigned>(rows), fa::cache::kCombineThreads, 0, cs, w,
                                           static_cast<T *>(o), lse, rows_block, rows);
                return second ? launched() : FA_ERR_CUDA;
            });
        };
        const auto with_rows = [&](auto warp_rows) {
            constexpr int ROWS = decltype(warp_rows)::value;
            using F = fa::cache4::Dec4Cfg<D, ROWS>;
            const long long blocks = std::min<long long>(static_cast<long long>(sms) * F::BLOCKS, fa::cache::kMaxBlocks);
            if (ROWS <= 8 && segments > blocks && bound <= std::min(kWholeUnits, kShortUnits + segments / blocks))
                return launch_short<D, ROWS>(w, segments, o, lse, dtype, cs);
            return run(F(), F::BLOCKS, [&](auto t, unsigned grid) {
                using T = decltype(t);
                return launch_dependent(decode_kernel<D, ROWS, T>(), grid, F::THREADS, F::SMEM, cs, w, static_cast<T *>(o), lse);
            });
        };
        if constexpr (D >= 96) {
            const auto on_tensor_cores = [&](auto group) {
                constexpr int ROWS = decltype(group)::value;
                using F = fa::cache4::Tc4Cfg<D, ROWS>;
                return run(F(), 1, [&](auto t, unsigned grid) {
                    using T = decltype(t);
                    return launch_dependent(fa::cache4::fa_cache4_tc_kernel<D, ROWS, T>, grid, F::THREADS, F::SMEM, cs, w,
                                            static_cast<T *>(o), lse);
                });
            };
            if (on_tcgen05<D>(w.R, segments, bound, sms)) {
                if constexpr (D == 128)
                    if (w.R <= 32)
                        return on_tensor_cores(Dim<32>());
                return on_tensor_cores(Dim<64>());
            }
        }
        return w.R <= 4 ? with_rows(Dim<4>()) : w.R <= 8 ? with_rows(Dim<8>()) : with_rows(Dim<16>());
    });
}

}  // extern "C"
