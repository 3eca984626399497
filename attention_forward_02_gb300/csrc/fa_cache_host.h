// fa_cache_host.h -- host-side pieces shared by the two paged caches (fa_cache.cu,
// fa_cache4.cu): checks of their arguments, the layout of query rows, launches.
// Internal, as fa_host.h is.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "fa.h"
#include "fa_host.h"

namespace fa_host {

constexpr int kMaxNq = 16;
constexpr int kMaxBatch = 65535;  // a grid's y and z extent

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
inline Shape shape_of(int R)
{
    if (R <= 8)
        return {1, 1, 8};
    const int row_warps = R <= 16 ? 1 : R <= 32 ? 2 : 4;
    return {2, row_warps, 16 * row_warps};
}

// Bytes of the plan at the workspace's start (a 64-bit number, and one a sequence).
inline size_t plan_bytes(int B) { return (static_cast<size_t>(B) + 2) / 2 * 16; }

inline uintptr_t u(const void *p) { return reinterpret_cast<uintptr_t>(p); }

struct Range {
    uintptr_t at;
    size_t bytes;
};

inline bool any_overlap(const Range &a, const Range *others, int count)
{
    for (int i = 0; i < count; ++i)
        if (a.at && others[i].at && a.bytes && others[i].bytes && overlaps(a.at, a.bytes, others[i].at, others[i].bytes))
            return true;
    return false;
}

// A stride: not negative, and what it spans small enough for the sums and byte counts here.
inline bool fine(long long s, int extent) { return s >= 0 && (extent <= 1 || s <= (1ll << 40) / (extent - 1)); }

inline fa_status_t check_batch(const int *seq_lens, const int *table, long long table_stride, int max_pages, int B, int page)
{
    if (!seq_lens || !table || max_pages < 1 || table_stride < max_pages || !fine(table_stride, B))
        return FA_ERR_INVALID_ARG;
    if (B > kMaxBatch || static_cast<long long>(max_pages) * page > 0x7fffffffLL)
        return FA_ERR_UNSUPPORTED;
    if ((u(seq_lens) | u(table)) & 3u)
        return FA_ERR_MISALIGNED;
    return FA_OK;
}

// Strides of an input with rows of d values, in elements.
inline bool strides_aligned(long long a, long long b, long long c = 0) { return ((a | b | c) & 7) == 0; }

// Checks of the queries of a decoding call or a selection over a cache of `heads` KV heads.
inline fa_status_t check_queries(int heads, int d, const void *q, long long &sb, long long &sh, long long &sr, int B,
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
    if (Hq % heads != 0 || !q || !fine(sb, B) || !fine(sh, Hq) || !fine(sr, Nq))
        return FA_ERR_INVALID_ARG;
    if (u(q) & 15u || !strides_aligned(sb, sh, sr))
        return FA_ERR_MISALIGNED;
    *r = {u(q), static_cast<size_t>((B - 1) * sb + (Hq - 1) * sh + (Nq - 1) * sr + d) * 2};
    return FA_OK;
}

// Launch of a kernel that may begin before the one ahead of it has ended (it
// waits for that one itself).  A launch that fails leaves no error for a later call to find.
template <typename... P, typename... A>
inline bool launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, const A &...args)
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
    if (cudaLaunchKernelEx(&cfg, kernel, P(args)...) == cudaSuccess)
        return true;
    cudaGetLastError();
    return false;
}

inline fa_status_t launched() { return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

template <int D>
struct Dim {
    static constexpr int value = D;
};
template <typename F>
fa_status_t by_dim(int d, F f)
{
    return d == 32 ? f(Dim<32>()) : d == 64 ? f(Dim<64>()) : d == 96 ? f(Dim<96>()) : f(Dim<128>());
}

}  // namespace fa_host
