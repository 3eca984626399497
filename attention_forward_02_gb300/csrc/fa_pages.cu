// fa_pages.cu -- host side of fa_cache_plan and fa_cache_trim declared in
// include/fa.h: argument checks and the launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <functional>
#include <mutex>

#include "fa.h"
#include "fa_cache_host.h"
#include "fa_host.h"
#include "fa_pages_kernel.cuh"

namespace {

using namespace fa_host;
using fa::pages::kMaxBatch;

struct PagesState {
    std::once_flag once;
    cudaError_t err = cudaErrorUnknown;
    unsigned int *status = nullptr;
};
PagesState g_pages[kMaxDevices];

void init_pages(PagesState &st)
{
    void *p = nullptr;
    st.err = cudaGetSymbolAddress(&p, fa::g_fa_status);
    st.status = static_cast<unsigned int *>(p);
    const int most = static_cast<int>(fa::pages::smem_bytes(kMaxBatch));
    const cudaFuncAttribute a = cudaFuncAttributeMaxDynamicSharedMemorySize;
    if (st.err == cudaSuccess)
        st.err = cudaFuncSetAttribute(fa::pages::fa_cache_plan_kernel, a, most);
    if (st.err == cudaSuccess)
        st.err = cudaFuncSetAttribute(fa::pages::fa_cache_trim_kernel, a, most);
}

fa_status_t device(PagesState **out)
{
    EncodeTiledFn encode = nullptr;
    const fa_status_t s = encoder(&encode, nullptr);
    if (s != FA_OK)
        return s;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        return FA_ERR_CUDA;
    PagesState &st = g_pages[dev];
    std::call_once(st.once, init_pages, std::ref(st));
    if (st.err != cudaSuccess)
        return FA_ERR_CUDA;
    *out = &st;
    return FA_OK;
}

// Checks that both calls share.
fa_status_t check(const int *ring, int num_pages, const long long *counts, const int *table, long long table_stride,
                  int max_pages, const int *lens, const int *other, const long long *out, int page, int B)
{
    if (num_pages < 1 || !ring || !counts || !table || !lens || !other || !out || max_pages < 1 || table_stride < max_pages ||
        !fine(table_stride, B))
        return FA_ERR_INVALID_ARG;
    if ((page != 16 && page != 32 && page != 64 && page != 128) || B > kMaxBatch ||
        static_cast<long long>(num_pages) * page > 0x7fffffffLL || static_cast<long long>(max_pages) * page > 0x7fffffffLL)
        return FA_ERR_UNSUPPORTED;
    if ((u(ring) | u(table) | u(lens) | u(other)) & 3u || (u(counts) | u(out)) & 7u)
        return FA_ERR_MISALIGNED;
    return FA_OK;
}

int log2_of(int page)
{
    int n = 4;
    while ((1 << n) < page)
        ++n;
    return n;
}

// `written` overlap neither one another nor `read`.
bool separate(const Range *written, int n, const Range *read, int m)
{
    for (int i = 0; i < n; ++i)
        if (any_overlap(written[i], written, i) || any_overlap(written[i], read, m))
            return false;
    return true;
}

}  // namespace

namespace fa_host {

unsigned int *pages_status_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, fa::g_fa_status) == cudaSuccess ? static_cast<unsigned int *>(p) : nullptr;
}

}  // namespace fa_host

extern "C" {

fa_status_t fa_cache_plan(const int *ring, int num_pages, const long long *counts, int *page_table,
                          long long table_stride, int max_pages, const int *seq_lens, const int *new_lens,
                          int *cu_seqlens, int *ends, int *positions, int *slots, long long *counts_out, int page, int B,
                          int T, void *stream)
{
    if (B < 0 || T < 0)
        return FA_ERR_INVALID_ARG;
    if (B == 0)
        return FA_OK;  // empty problem
    fa_status_t s = check(ring, num_pages, counts, page_table, table_stride, max_pages, seq_lens, new_lens, counts_out,
                          page, B);
    if (s != FA_OK)
        return s;
    if (!cu_seqlens || !ends || (T > 0 && (!positions || !slots)))
        return FA_ERR_INVALID_ARG;
    if ((u(cu_seqlens) | u(ends) | u(positions) | u(slots)) & 3u)
        return FA_ERR_MISALIGNED;
    const size_t table = (static_cast<size_t>(B - 1) * table_stride + max_pages) * 4, lens = static_cast<size_t>(B) * 4;
    const Range written[6] = {{u(page_table), table},
                              {u(cu_seqlens), lens + 4},
                              {u(ends), lens},
                              {u(positions), static_cast<size_t>(T) * 4},
                              {u(slots), static_cast<size_t>(T) * 4},
                              {u(counts_out), 16}};
    const Range read[4] = {{u(ring), static_cast<size_t>(num_pages) * 4},
                           {u(seq_lens), lens},
                           {u(new_lens), lens},
                           {counts == counts_out ? 0 : u(counts), 16}};
    if (!separate(written, 6, read, 4))
        return FA_ERR_INVALID_ARG;
    PagesState *st = nullptr;
    if ((s = device(&st)) != FA_OK)
        return s;
    using namespace fa::pages;
    const Pool pool = {const_cast<int *>(ring), num_pages, counts, counts_out};
    const Lengths in = {seq_lens, new_lens, B, log2_of(page)};
    const Rows rows = {positions, slots, T};
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (!launch_dependent(fa_cache_plan_kernel, 1, kThreads, smem_bytes(B), cs, pool, in, page_table, table_stride, max_pages,
                          cu_seqlens, ends, rows, st->status))
        return FA_ERR_CUDA;
    constexpr int kPerBlock = kRowThreads * kRows;
    const unsigned blocks = static_cast<unsigned>((static_cast<long long>(T) + kPerBlock - 1) / kPerBlock);
    if (T > kOwnRows && !launch_dependent(fa_cache_rows_kernel, blocks, kRowThreads, 0, cs, in, page_table, table_stride,
                                          num_pages, cu_seqlens, ends, rows, st->status))
        return FA_ERR_CUDA;
    return launched();
}

fa_status_t fa_cache_trim(int *ring, int num_pages, const long long *counts, const int *page_table,
                          long long table_stride, int max_pages, const int *seq_lens, const int *keep_lens,
                          long long *counts_out, int page, int B, void *stream)
{
    if (B < 0)
        return FA_ERR_INVALID_ARG;
    if (B == 0)
        return FA_OK;  // empty problem
    fa_status_t s = check(ring, num_pages, counts, page_table, table_stride, max_pages, seq_lens, keep_lens, counts_out,
                          page, B);
    if (s != FA_OK)
        return s;
    const size_t lens = static_cast<size_t>(B) * 4;
    const Range written[2] = {{u(ring), static_cast<size_t>(num_pages) * 4}, {u(counts_out), 16}};
    const Range read[4] = {{u(page_table), (static_cast<size_t>(B - 1) * table_stride + max_pages) * 4},
                           {u(seq_lens), lens},
                           {u(keep_lens), lens},
                           {counts == counts_out ? 0 : u(counts), 16}};
    if (!separate(written, 2, read, 4))
        return FA_ERR_INVALID_ARG;
    PagesState *st = nullptr;
    if ((s = device(&st)) != FA_OK)
        return s;
    using namespace fa::pages;
    const Pool pool = {ring, num_pages, counts, counts_out};
    const Lengths in = {seq_lens, keep_lens, B, log2_of(page)};
    return launch_dependent(fa_cache_trim_kernel, 1, kThreads, smem_bytes(B), static_cast<cudaStream_t>(stream), pool,
                            in, page_table, table_stride, max_pages, st->status)
               ? launched()
               : FA_ERR_CUDA;
}

}  // extern "C"
