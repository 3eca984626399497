// fa_cache.cu -- host side of the 8-bit paged KV cache declared in include/fa.h:
// argument checks and the launches of writing, reading back, page selection
// and decoding attention.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <functional>
#include <mutex>

#include "fa.h"
#include "fa_cache_decode_kernel.cuh"
#include "fa_cache_kernel.cuh"
#include "fa_host.h"

namespace {

using fa::cache::Batch;
using fa::cache::Cache;
using fa::cache::Queries;
using fa_host::kMaxDevices;
using fa_host::overlaps;

constexpr int kMaxNq = 16;
constexpr int kMaxBatch = 65535;  // a grid's y and z extent
// Units of a segment that one block may take whole: one launch in place of two,
// but the units one after the other.  8 KV heads, e4m3, whole / shared out, us on the
// GPU (in a graph):
//                      1 unit     4 units     8 units     16 units
//   d = 128, 1 seq.    4.6 / 6.6  6.2 / 7.4   8.4 / 7.7   13.0 / 8.0
//            16                   6.6 / 8.7   8.8 / 10.9
//            56                   8.5 / 15.8  13.0 / 21.7
//   d = 64,  1         4.1 / 6.0  5.7 / 6.9   8.0 / 7.2
//            16                   6.3 / 8.0   8.5 / 9.9
//            56                   7.9 / 13.2  11.4 / 18.3
// As called from Python one sequence takes 8.9 / 11 us at 1 to 8 units.  So eight units
// of few segments are where a captured call loses (0.7 us); all else gains.
constexpr long long kWholeUnits = 8;

struct CacheState {
    std::once_flag once;
    cudaError_t err = cudaErrorUnknown;
    unsigned int *status = nullptr;
};
CacheState g_cache[kMaxDevices];

// The decoding kernel: warps of 8 or 16 query rows, one 16-key tile at a time or,
// where stages hold 128 keys (d <= 64), two (8 x 8,000 keys of 32 heads of 64: 32 us
// against 37).
template <int D, int NT, typename T, typename C>
constexpr auto decode_kernel()
{
    return fa::cache::fa_cache_decode_kernel<D, NT, D <= 64 ? 2 : 1, T, C>;
}

template <int D, int NT>
cudaError_t set_smem_attr()
{
    using namespace fa::cache;
    const cudaFuncAttribute a = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t e = cudaFuncSetAttribute(decode_kernel<D, NT, __half, E4M3>(), a, DecCfg<D>::SMEM);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(decode_kernel<D, NT, __half, I8>(), a, DecCfg<D>::SMEM);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(decode_kernel<D, NT, __nv_bfloat16, E4M3>(), a, DecCfg<D>::SMEM);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(decode_kernel<D, NT, __nv_bfloat16, I8>(), a, DecCfg<D>::SMEM);
    return e;
}

template <int D>
cudaError_t set_smem_attrs()
{
    const cudaError_t e = set_smem_attr<D, 1>();
    return e == cudaSuccess ? set_smem_attr<D, 2>() : e;
}

void init_cache(CacheState &st)
{
    void *p = nullptr;
    st.err = cudaGetSymbolAddress(&p, fa::g_fa_status);
    st.status = static_cast<unsigned int *>(p);
    if (st.err == cudaSuccess) st.err = set_smem_attrs<32>();
    if (st.err == cudaSuccess) st.err = set_smem_attrs<64>();
    if (st.err == cudaSuccess) st.err = set_smem_attrs<96>();
    if (st.err == cudaSuccess) st.err = set_smem_attrs<128>();
}

// How the R query rows of a KV head are laid out: tiles of 8 rows a warp, warps of
// a block along the rows (the others take keys), rows a block.  Rows beyond 64 go
// to further row groups, which read the codes again.
// Sixteen rows a warp share one conversion of the codes, where two warps of eight
// convert them twice; they need Q in shared memory.  16 x 16,384 keys (mean 8,700)
// of 8 heads, sixteen a warp against eight: 16 rows, d = 128, int8 83 / 89 us, e4m3
// 82 / 75; d = 64 47 / 55 and 44 / 47; 64 rows, d = 128 233 / 285 and 216 / 229,
// d = 64 126 / 177 and 113 / 142.  Up to 8 rows the second eight would be padding.
struct Shape {
    int tiles, row_warps, rows_block;
};
Shape shape_of(int R)
{
    if (R <= 8)
        return {1, 1, 8};
    const int row_warps = R <= 16 ? 1 : R <= 32 ? 2 : 4;
    return {2, row_warps, 16 * row_warps};
}

// A code buffer as [num_pages * heads, page, d] bytes: boxes of `box` rows of
// `width` columns, each row swizzled by its width.
fa_status_t encode_codes(fa_host::EncodeTiledFn encode, CUtensorMap *map, void *codes, const fa_cache_t *c, int width,
                         int box)
{
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c->d), static_cast<cuuint64_t>(c->page),
                                static_cast<cuuint64_t>(c->num_pages) * c->heads};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(c->d), static_cast<cuuint64_t>(c->page) * c->d};
    const cuuint32_t extent[3] = {static_cast<cuuint32_t>(width), static_cast<cuuint32_t>(box), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUtensorMapSwizzle swizzle = width == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                       : width == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                     : CU_TENSOR_MAP_SWIZZLE_32B;
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, codes, dims, strides, extent, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? FA_OK
               : FA_ERR_CUDA;
}

// Bytes of the plan at the workspace's start (a 64-bit number, and one a sequence).
size_t plan_bytes(int B) { return (static_cast<size_t>(B) + 2) / 2 * 16; }

// The current device's status word and SM count.
fa_status_t device(CacheState **out, int *num_sms, fa_host::EncodeTiledFn *encoder = nullptr)
{
    fa_host::EncodeTiledFn encode = nullptr;
    const fa_status_t s = fa_host::encoder(&encode, num_sms);
    if (encoder)
        *encoder = encode;
    if (s != FA_OK)
        return s;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        return FA_ERR_CUDA;
    CacheState &st = g_cache[dev];
    std::call_once(st.once, init_cache, std::ref(st));
    if (st.err != cudaSuccess)
        return FA_ERR_CUDA;
    *out = &st;
    return FA_OK;
}

uintptr_t u(const void *p) { return reinterpret_cast<uintptr_t>(p); }

struct Range {
    uintptr_t at;
    size_t bytes;
};

bool any_overlap(const Range &a, const Range *others, int count)
{
    for (int i = 0; i < count; ++i)
        if (a.at && others[i].at && a.bytes && others[i].bytes && overlaps(a.at, a.bytes, others[i].at, others[i].bytes))
            return true;
    return false;
}

// Checks of a cache that need no device; fills its six buffers' ranges.
constexpr int kCacheRanges = 6;
fa_status_t check_cache(const fa_cache_t *c, Range (&r)[kCacheRanges])
{
    if (!c || c->num_pages < 1 || c->heads < 1)
        return FA_ERR_INVALID_ARG;
    if (static_cast<long long>(c->num_pages) * c->heads > 0x7fffffffLL)
        return FA_ERR_UNSUPPORTED;
    if ((c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) ||
        (c->d != 32 && c->d != 64 && c->d != 96 && c->d != 128) || (c->format != FA_E4M3 && c->format != FA_INT8) ||
        c->heads > kMaxBatch / 2)
        return FA_ERR_UNSUPPORTED;
    if (!c->k || !c->v || !c->k_scale || !c->v_scale || (c->k_mean == nullptr) != (c->k_mean_scale == nullptr))
        return FA_ERR_INVALID_ARG;
    if ((u(c->k) | u(c->v) | u(c->k_mean)) & 15u || (u(c->k_scale) | u(c->v_scale) | u(c->k_mean_scale)) & 3u)
        return FA_ERR_MISALIGNED;
    const size_t ph = static_cast<size_t>(c->num_pages) * c->heads;
    r[0] = {u(c->k), ph * c->page * c->d};
    r[1] = {u(c->v), ph * c->page * c->d};
    r[2] = {u(c->k_scale), ph * 4};
    r[3] = {u(c->v_scale), ph * 4};
    r[4] = {u(c->k_mean), ph * c->d};
    r[5] = {u(c->k_mean_scale), ph * 4};
    for (int i = 0; i < kCacheRanges; ++i)
        if (any_overlap(r[i], r, i))
            return FA_ERR_INVALID_ARG;
    return FA_OK;
}

fa_status_t check_batch(const int *seq_lens, const int *table, long long table_stride, int max_pages, int B, int page)
{
    if (!seq_lens || !table || max_pages < 1 || table_stride < max_pages)
        return FA_ERR_INVALID_ARG;
    if (B > kMaxBatch || static_cast<long long>(max_pages) * page > 0x7fffffffLL)
        return FA_ERR_UNSUPPORTED;
    if ((u(seq_lens) | u(table)) & 3u)
        return FA_ERR_MISALIGNED;
    return FA_OK;
}

Cache device_cache(const fa_cache_t *c)
{
    int log2_page = 4;
    while ((1 << log2_page) < c->page)
        ++log2_page;
    return {static_cast<uint8_t *>(c->k), static_cast<uint8_t *>(c->v), c->k_scale, c->v_scale,
            reinterpret_cast<int8_t *>(c->k_mean), c->k_mean_scale, c->num_pages, c->heads, c->page, log2_page};
}

// Strides of an input with rows of d values, in elements.
bool strides_ok(long long a, long long b, long long c = 0) { return a >= 0 && b >= 0 && c >= 0; }
bool strides_aligned(long long a, long long b, long long c = 0) { return ((a | b | c) & 7) == 0; }

// Checks of the queries of fa_decode_cache and fa_cache_select.
fa_status_t check_queries(const fa_cache_t *cache, const void *q, long long &sb, long long &sh, long long &sr, int B,
                          int Hq, int Nq, int causal, fa_dtype_t dtype, Range *r)
{
    sb = B == 1 ? 0 : sb;  // the stride of a dimension of one means nothing
    sh = Hq == 1 ? 0 : sh;
    sr = Nq == 1 ? 0 : sr;
    if (causal != 0 && causal != 1)
        return FA_ERR_INVALID_ARG;
    if (dtype != FA_FP16 && dtype != FA_BF16)
        return FA_ERR_UNSUPPORTED;
    if (Nq < 1 || Nq > kMaxNq)
        return FA_ERR_UNSUPPORTED;
    if (Hq % cache->heads != 0 || !q || !strides_ok(sb, sh, sr))
        return FA_ERR_INVALID_ARG;
    if (u(q) & 15u || !strides_aligned(sb, sh, sr))
        return FA_ERR_MISALIGNED;
    *r = {u(q), static_cast<size_t>((B - 1) * sb + (Hq - 1) * sh + (Nq - 1) * sr + cache->d) * 2};
    return FA_OK;
}

// Launch of a kernel that may begin before the one ahead of it has ended (it
// waits for that one itself).
template <typename... P, typename... A>
bool launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, const A &...args)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...) == cudaSuccess;
}

fa_status_t launched() { return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// f(T, C) with the 16-bit type and the code type.
template <typename F>
fa_status_t by_types(fa_dtype_t dtype, int format, F f)
{
    if (dtype == FA_FP16)
        return format == FA_E4M3 ? f(__half(), fa::cache::E4M3()) : f(__half(), fa::cache::I8());
    return format == FA_E4M3 ? f(__nv_bfloat16(), fa::cache::E4M3()) : f(__nv_bfloat16(), fa::cache::I8());
}

template <int D>
struct Dim {
    static constexpr int value = D;
};
template <typename F>
fa_status_t by_dim(int d, F f)
{
    return d == 32 ? f(Dim<32>()) : d == 64 ? f(Dim<64>()) : d == 96 ? f(Dim<96>()) : f(Dim<128>());
}

}  // namespace

namespace fa_host {

fa_status_t take_cache_status(unsigned int *word)
{
    *word = 0;
    const unsigned int zero = 0;
    if (cudaMemcpyFromSymbol(word, fa::g_fa_status, sizeof(*word)) != cudaSuccess)
        return FA_ERR_CUDA;
    if (cudaMemcpyToSymbol(fa::g_fa_status, &zero, sizeof(zero)) != cudaSuccess)
        return FA_ERR_CUDA;
    return FA_OK;
}

}  // namespace fa_host

extern "C" {

fa_status_t fa_cache_write(const fa_cache_t *cache, const void *k, const void *v, long long k_token_stride,
                           long long k_head_stride, long long v_token_stride, long long v_head_stride,
                           const int *cu_seqlens, const int *seq_lens, const int *page_table, long long table_stride,
                           int max_pages, int B, int T, fa_dtype_t dtype, void *stream)
{
    Range own[kCacheRanges];
    fa_status_t s = check_cache(cache, own);
    if (s != FA_OK)
        return s;
    if (B < 0 || T < 0)
        return FA_ERR_INVALID_ARG;
    if (dtype != FA_FP16 && dtype != FA_BF16)
        return FA_ERR_UNSUPPORTED;
    if (B == 0 || T == 0)
        return FA_OK;  // empty problem
    if ((s = check_batch(seq_lens, page_table, table_stride, max_pages, B, cache->page)) != FA_OK)
        return s;
    if (T == 1)  // the stride of a dimension of one means nothing
        k_token_stride = v_token_stride = 0;
    if (cache->heads == 1)
        k_head_stride = v_head_stride = 0;
    if (!k || !v || !strides_ok(k_token_stride, k_head_stride) || !strides_ok(v_token_stride, v_head_stride) ||
        (!cu_seqlens && T % B != 0))
        return FA_ERR_INVALID_ARG;
    if ((u(k) | u(v)) & 15u || u(cu_seqlens) & 3u || !strides_aligned(k_token_stride, k_head_stride) ||
        !strides_aligned(v_token_stride, v_head_stride))
        return FA_ERR_MISALIGNED;
    const Range in[5] = {
        {u(k), static_cast<size_t>((T - 1) * k_token_stride + (cache->heads - 1) * k_head_stride + cache->d) * 2},
        {u(v), static_cast<size_t>((T - 1) * v_token_stride + (cache->heads - 1) * v_head_stride + cache->d) * 2},
        {u(seq_lens), static_cast<size_t>(B) * 4},
        {u(cu_seqlens), (static_cast<size_t>(B) + 1) * 4},
        {u(page_table), (static_cast<size_t>(B - 1) * table_stride + max_pages) * 4}};
    for (const Range &r : own)
        if (any_overlap(r, in, 5))
            return FA_ERR_INVALID_ARG;
    CacheState *st = nullptr;
    if ((s = device(&st, nullptr)) != FA_OK)
        return s;
    const Cache c = device_cache(cache);
    const Batch batch = {seq_lens, page_table, table_stride, max_pages, cache->num_pages, st->status};
    const fa::cache::NewRows rows = {{k, v},
                                     {k_token_stride, v_token_stride},
                                     {k_head_stride, v_head_stride},
                                     cu_seqlens,
                                     cu_seqlens ? 0 : T / B,
                                     T,
                                     B};
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    // A warp a sequence, head, and of K and V.  The totals decide, so that a batch whose
    // rows are nearly all one sequence's is slow on either side: a prompt of 512 rows
    // takes 114 us in 512 slots (one warp a head walks it), 48 in 511 (every block of the
    // other kernel counts over the slots), and 4.4 alone (8 heads of 128, e4m3).
    if (T <= B) {
        const long long units = 2ll * B * cache->heads;
        if (units > 0x7fffffffLL)
            return FA_ERR_UNSUPPORTED;
        const unsigned blocks = static_cast<unsigned>((units + fa::cache::kStepWarps - 1) / fa::cache::kStepWarps);
        return by_types(dtype, cache->format, [&](auto t, auto code) {
            fa::cache::fa_cache_step_kernel<decltype(t), decltype(code)>
                <<<blocks, 32 * fa::cache::kStepWarps, 0, cs>>>(c, batch, rows, cache->d);
            return launched();
        });
    }
    // a block a touched page, of which there are at most T / page + 2 B however the
    // rows are spread over the sequences
    const long long pages = T / cache->page + 2ll * B;
    if (pages > 0x7fffffffLL)
        return FA_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(pages), 2 * cache->heads);
    const int threads = (cache->page / fa::cache::kWriteRows * (cache->d / 8) + 31) / 32 * 32;
    return by_types(dtype, cache->format, [&](auto t, auto code) {
        fa::cache::fa_cache_write_kernel<decltype(t), decltype(code)><<<grid, threads, 0, cs>>>(c, batch, rows, cache->d);
        return launched();
    });
}

fa_status_t fa_cache_read(const fa_cache_t *cache, void *k, void *v, const int *seq_lens, const int *page_table,
                          long long table_stride, int max_pages, int B, int N, fa_dtype_t dtype, void *stream)
{
    Range own[kCacheRanges];
    fa_status_t s = check_cache(cache, own);
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
    constexpr int kPerBlock = fa::cache::kReadThreads * fa::cache::kReadSteps;
    const long long chunks = (static_cast<long long>(N) * (cache->d / 16) + kPerBlock - 1) / kPerBlock;
    const long long blocks = chunks * B * cache->heads;
    if (blocks > 0x7fffffffLL)
        return FA_ERR_UNSUPPORTED;
    const size_t bytes = static_cast<size_t>(B) * cache->heads * N * cache->d * 2;
    const Range out[2] = {{u(k), bytes}, {u(v), bytes}};
    const Range in[2] = {{u(seq_lens), static_cast<size_t>(B) * 4},
                         {u(page_table), (static_cast<size_t>(B - 1) * table_stride + max_pages) * 4}};
    if (any_overlap(out[0], own, kCacheRanges) || any_overlap(out[1], own, kCacheRanges) || any_overlap(out[0], in, 2) ||
        any_overlap(out[1], in, 2) || any_overlap(out[0], out + 1, 1))
        return FA_ERR_INVALID_ARG;
    CacheState *st = nullptr;
    if ((s = device(&st, nullptr)) != FA_OK)
        return s;
    const Cache c = device_cache(cache);
    const Batch batch = {seq_lens, page_table, table_stride, max_pages, cache->num_pages, st->status};
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return by_types(dtype, cache->format, [&](auto t, auto code) {
        using T = decltype(t);
        fa::cache::fa_cache_read_kernel<T, decltype(code)>
            <<<dim3(static_cast<unsigned>(blocks), 2), fa::cache::kReadThreads, 0, cs>>>(
                c, batch, static_cast<T *>(k), static_cast<T *>(v), N, cache->d, static_cast<int>(chunks));
        return launched();
    });
}

size_t fa_decode_cache_workspace_size(int B, int Hq, int Hkv, int Nq, int d)
{
    if (B < 0 || Hq < 0 || Hkv < 1 || Hq % Hkv != 0 || Nq < 1 || Nq > kMaxNq ||
        (d != 32 && d != 64 && d != 96 && d != 128))
        return 0;
    const int rows_block = shape_of(Hq / Hkv * Nq).rows_block;
    return plan_bytes(B) + static_cast<size_t>(2 * fa::cache::kMaxBlocks) * rows_block * (d + 2) * 4;
}

fa_status_t fa_decode_cache(const fa_cache_t *cache, const void *q, long long q_batch_stride, long long q_head_stride,
                            long long q_row_stride, void *o, float *lse, const int *seq_lens, const int *page_table,
                            long long table_stride, int max_pages, const int *pages, int slots, void *workspace,
                            size_t workspace_bytes, int B, int Hq, int Nq, float scale, int causal, fa_dtype_t dtype,
                            void *stream)
{
    Range own[kCacheRanges];
    fa_status_t s = check_cache(cache, own);
    if (s != FA_OK)
        return s;
    if (B < 0 || Hq < 0 || !std::isfinite(scale) || (pages && slots < 1))
        return FA_ERR_INVALID_ARG;
    if (scale < 0.f)
        return FA_ERR_UNSUPPORTED;
    if (B == 0 || Hq == 0)
        return FA_OK;  // empty problem
    if ((s = check_batch(seq_lens, page_table, table_stride, max_pages, B, cache->page)) != FA_OK)
        return s;
    Range in[4];
    if ((s = check_queries(cache, q, q_batch_stride, q_head_stride, q_row_stride, B, Hq, Nq, causal, dtype, in)) != FA_OK)
        return s;
    const size_t need = fa_decode_cache_workspace_size(B, Hq, cache->heads, Nq, cache->d);
    if (!o || !workspace || workspace_bytes < need)
        return FA_ERR_INVALID_ARG;
    if ((u(o) | u(workspace)) & 15u || (u(lse) | u(pages)) & 3u)
        return FA_ERR_MISALIGNED;
    const long long rows = static_cast<long long>(B) * Hq * Nq;
    if (rows > 0x7fffffffLL)
        return FA_ERR_UNSUPPORTED;
    in[1] = {u(seq_lens), static_cast<size_t>(B) * 4};
    in[2] = {u(page_table), (static_cast<size_t>(B - 1) * table_stride + max_pages) * 4};
    in[3] = {u(pages), static_cast<size_t>(B) * cache->heads * Nq * slots * 4};
    const Range out[3] = {{u(o), static_cast<size_t>(rows) * cache->d * 2},
                          {u(lse), static_cast<size_t>(rows) * 4},
                          {u(workspace), need}};
    for (int i = 0; i < 3; ++i)
        if (any_overlap(out[i], own, kCacheRanges) || any_overlap(out[i], in, 4) || any_overlap(out[i], out, i))
            return FA_ERR_INVALID_ARG;
    CacheState *st = nullptr;
    int sms = 0;
    fa_host::EncodeTiledFn encode = nullptr;
    if ((s = device(&st, &sms, &encode)) != FA_OK)
        return s;
    const Cache c = device_cache(cache);
    const Batch batch = {seq_lens, page_table, table_stride, max_pages, cache->num_pages, st->status};
    const Queries qs = {q, q_batch_stride, q_head_stride, q_row_stride, Hq / cache->heads, Nq, causal};
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    fa::cache::Work w = {};
    w.cache = c;
    w.batch = batch;
    w.q = qs;
    w.pages = pages;
    w.slots = slots;
    w.B = B;
    w.R = qs.G * (pages ? 1 : Nq);
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
    const int step = cache->d <= 64 ? fa::cache::DecCfg<64>::STEP : fa::cache::DecCfg<128>::STEP;
    const int box = cache->page < step ? cache->page : step;
    w.log2_box = box == 128 ? 7 : box == 64 ? 6 : box == 32 ? 5 : 4;
    fa::cache::Maps maps = {};
    const int width[2] = {cache->d == 96 ? 64 : cache->d, 32};
    for (int i = 0; i < (cache->d == 96 ? 2 : 1); ++i)
        if ((s = encode_codes(encode, &maps.k[i], cache->k, cache, width[i], box)) != FA_OK ||
            (s = encode_codes(encode, &maps.v[i], cache->v, cache, width[i], box)) != FA_OK)
            return s;
    const long long segments = static_cast<long long>(B) * (pages ? Nq : 1) * cache->heads * w.groups;
    const long long keys = static_cast<long long>(pages && slots < max_pages ? slots : max_pages) * cache->page;
    const long long units = (keys - 1) / step + 1;  // of a segment, at most
    const long long resident =
        static_cast<long long>(sms) * (cache->d == 32 ? fa::cache::DecCfg<32>::BLOCKS : fa::cache::DecCfg<128>::BLOCKS);
    long long blocks = resident < fa::cache::kMaxBlocks ? resident : fa::cache::kMaxBlocks;
    w.whole = units <= kWholeUnits && segments <= blocks;
    if (w.whole)
        blocks = segments;
    else if (segments * units < blocks)
        blocks = segments * units;
    return by_dim(cache->d, [&](auto dim) {
        return by_types(dtype, cache->format, [&](auto t, auto code) {
            constexpr int D = decltype(dim)::value;
            using T = decltype(t);
            using C = decltype(code);
            const bool first = launch_dependent(
                shape.tiles == 1 ? decode_kernel<D, 1, T, C>() : decode_kernel<D, 2, T, C>(),
                static_cast<unsigned>(blocks), fa::cache::kDecThreads, fa::cache::DecCfg<D>::SMEM, cs, maps, w,
                static_cast<T *>(o), lse);
            if (!first)
                return FA_ERR_CUDA;
            if (w.whole)
                return launched();
            // parts of a segment, on average: a warp takes a few of them alone (32 x 2
            // queries of 4 heads: 5.5 us against 8.0 with four warps a row), four share
            // many (57 a segment at one sequence of 131,072 keys: 6.1 us against 9)
            constexpr int kWarps = fa::cache::kCombineThreads / 32;
            const bool second =
                blocks <= segments * fa::cache::kCombineEach
                    ? launch_dependent(fa::cache::fa_cache_combine_kernel<D, T, 1>,
                                       static_cast<unsigned>((rows + kWarps - 1) / kWarps), fa::cache::kCombineThreads, 0,
                                       cs, w, static_cast<T *>(o), lse, rows_block, rows)
                    : launch_dependent(fa::cache::fa_cache_combine_kernel<D, T, kWarps>, static_cast<unsigned>(rows),
                                       fa::cache::kCombineThreads, 0, cs, w, static_cast<T *>(o), lse,
                                       rows_block, rows);
            if (!second)
                return FA_ERR_CUDA;
            return launched();
        });
    });
}

size_t fa_cache_select_workspace_size(int B, int Hkv, int Nq, int max_pages)
{
    if (B < 0 || Hkv < 1 || Nq < 1 || Nq > kMaxNq || max_pages < 1)
        return 0;
    return static_cast<size_t>(B) * Hkv * Nq * max_pages * 4;
}

fa_status_t fa_cache_select(const fa_cache_t *cache, const void *q, long long q_batch_stride, long long q_head_stride,
                            long long q_row_stride, const int *seq_lens, const int *page_table, long long table_stride,
                            int max_pages, int *pages, int slots, int keep_first, int keep_last, void *workspace,
                            size_t workspace_bytes, int B, int Hq, int Nq, int causal, fa_dtype_t dtype, void *stream)
{
    Range own[kCacheRanges];
    fa_status_t s = check_cache(cache, own);
    if (s != FA_OK)
        return s;
    if (!cache->k_mean || B < 0 || Hq < 0 || keep_first < 0 || keep_last < 1 ||
        static_cast<long long>(keep_first) + keep_last > slots)
        return FA_ERR_INVALID_ARG;
    if (B == 0 || Hq == 0)
        return FA_OK;  // empty problem
    if ((s = check_batch(seq_lens, page_table, table_stride, max_pages, B, cache->page)) != FA_OK)
        return s;
    Range in[3];
    if ((s = check_queries(cache, q, q_batch_stride, q_head_stride, q_row_stride, B, Hq, Nq, causal, dtype, in)) != FA_OK)
        return s;
    const size_t need = fa_cache_select_workspace_size(B, cache->heads, Nq, max_pages);
    if (!pages || !workspace || workspace_bytes < need)
        return FA_ERR_INVALID_ARG;
    if (u(workspace) & 15u || u(pages) & 3u)
        return FA_ERR_MISALIGNED;
    const long long segments = static_cast<long long>(B) * cache->heads * Nq;
    if (segments > 0x7fffffffLL)
        return FA_ERR_UNSUPPORTED;
    in[1] = {u(seq_lens), static_cast<size_t>(B) * 4};
    in[2] = {u(page_table), (static_cast<size_t>(B - 1) * table_stride + max_pages) * 4};
    const Range out[2] = {{u(pages), static_cast<size_t>(segments) * slots * 4}, {u(workspace), need}};
    for (int i = 0; i < 2; ++i)
        if (any_overlap(out[i], own, kCacheRanges) || any_overlap(out[i], in, 3) || any_overlap(out[i], out, i))
            return FA_ERR_INVALID_ARG;
    CacheState *st = nullptr;
    if ((s = device(&st, nullptr)) != FA_OK)
        return s;
    const Cache c = device_cache(cache);
    const Batch batch = {seq_lens, page_table, table_stride, max_pages, cache->num_pages, st->status};
    const Queries qs = {q, q_batch_stride, q_head_stride, q_row_stride, Hq / cache->heads, Nq, causal};
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    uint32_t *scores = static_cast<uint32_t *>(workspace);
    const dim3 grid((max_pages + fa::cache::kScorePages - 1) / fa::cache::kScorePages, cache->heads, B);
    s = by_dim(cache->d, [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        const bool ok = dtype == FA_FP16
                            ? launch_dependent(fa::cache::fa_cache_score_kernel<D, __half>, grid,
                                               fa::cache::kScoreThreads, 0, cs, c, batch, qs, scores, slots)
                            : launch_dependent(fa::cache::fa_cache_score_kernel<D, __nv_bfloat16>, grid,
                                               fa::cache::kScoreThreads, 0, cs, c, batch, qs, scores, slots);
        return ok ? FA_OK : FA_ERR_CUDA;
    });
    if (s != FA_OK)
        return s;
    using namespace fa::cache;
    const auto pick = [&](auto kernel, int threads) {
        return launch_dependent(kernel, static_cast<unsigned>(segments), threads, 0, cs, c, batch, qs, scores, pages, slots,
                                keep_first, keep_last);
    };
    if (!(max_pages <= kPickFew ? pick(fa_cache_pick_kernel<kPickFewThreads, kPickFew>, kPickFewThreads)
                                : pick(fa_cache_pick_kernel<kPickThreads, kPickHeld>, kPickThreads)))
        return FA_ERR_CUDA;
    return launched();
}

}  // extern "C"
